// torch_calls.cpp -- the Python binding's hot calls: checks of the tensors,
// allocation of what is not given, the current stream, and the call of
// libdecattn's C ABI, in one native step per call.
//
// A decode step's smallest kernels take 3 to 5 us; the same marshalling in
// Python takes 17 to 27 us a call.  The functions here take their arguments by
// position (binding.py names them) and return the result, or the library's
// status as an int where it is not DECATTN_OK.  No computation happens here.
#include <Python.h>

#include <dlfcn.h>

#include <optional>
#include <string>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "decattn.h"

namespace {

using at::ScalarType;
using at::Tensor;

// The library's entry points, by name (open() fills them).
#define DECATTN_CALLS(X)                                                                     \
  X(paged_plan) X(gqa_rope_append) X(gqa_rope_append_fp8kv) X(gqa_prefill)                   \
  X(gqa_prefill_fp8kv) X(gqa_prefill_plan_splits) X(gqa_prefill_workspace_size)              \
  X(gqa_decode) X(gqa_decode_fp8kv) X(gqa_decode_window) X(gqa_decode_fp8kv_window)          \
  X(gqa_decode_sinks) X(gqa_decode_fp8kv_sinks) X(gqa_decode_plan_splits)                    \
  X(gqa_decode_fp8kv_plan_splits) X(gqa_decode_sinks_plan_splits)                            \
  X(gqa_decode_workspace_size) X(gqa_decode_blocks) X(gqa_decode_fp8kv_blocks)               \
  X(gqa_decode_blocks_plan_splits) X(gqa_decode_weights) X(gqa_decode_fp8kv_weights)         \
  X(gqa_decode_weights_workspace_size) X(gqa_decode_weights_plan_splits)                     \
  X(gqa_block_bounds) X(gqa_select_blocks)              \
  X(gqa_select_workspace_size) X(gqa_kv_evict)
struct Library {
#define DECATTN_FIELD(name) decltype(&::name) name = nullptr;
  DECATTN_CALLS(DECATTN_FIELD)
#undef DECATTN_FIELD
} lib;

// A refusal: raised as the Python exception `type`.
struct Refused {
  PyObject* type;
  std::string what;
};
[[noreturn]] void type_error(const std::string& what) { throw Refused{PyExc_TypeError, what}; }
[[noreturn]] void value_error(const std::string& what) { throw Refused{PyExc_ValueError, what}; }

const char* name_of(ScalarType t) {
  switch (t) {
    case ScalarType::Int: return "torch.int32";
    case ScalarType::Long: return "torch.int64";
    case ScalarType::Byte: return "torch.uint8";
    case ScalarType::Half: return "torch.float16";
    case ScalarType::BFloat16: return "torch.bfloat16";
    case ScalarType::Float: return "torch.float32";
    case ScalarType::Double: return "torch.float64";
    case ScalarType::Float8_e4m3fn: return "torch.float8_e4m3fn";
    default: return c10::toString(t);
  }
}

std::string shape_of(const Tensor& t) {
  std::string s = "(";
  for (int64_t k = 0; k < t.dim(); ++k) s += (k ? ", " : "") + std::to_string(t.size(k));
  return s + ")";
}

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a torch.Tensor");
  return THPVariable_Unpack(o);
}

const Tensor& check(PyObject* o, const char* name, ScalarType type, int64_t dims) {
  const Tensor& t = tensor(o, name);
  if (t.scalar_type() != type)
    type_error(std::string(name) + ": expected " + name_of(type) + ", got " +
               name_of(t.scalar_type()));
  if (dims >= 0 && t.dim() != dims)
    value_error(std::string(name) + ": expected " + std::to_string(dims) + " dims, got shape " +
                shape_of(t));
  if (!t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
  return t;
}

// An 8-bit cache: uint8 or float8_e4m3fn (the same bytes).
const Tensor& check_codes(PyObject* o, const char* name) {
  const Tensor& t = tensor(o, name);
  return check(o, name,
               t.scalar_type() == ScalarType::Float8_e4m3fn ? ScalarType::Float8_e4m3fn
                                                            : ScalarType::Byte,
               4);
}

// fp16 / bf16 as the library numbers them.
int dtype16(const Tensor& t, const char* name) {
  if (t.scalar_type() == ScalarType::Half) return DECATTN_FP16;
  if (t.scalar_type() == ScalarType::BFloat16) return DECATTN_BF16;
  type_error(std::string(name) + " must be float16 or bfloat16");
}

int cuda_index(const Tensor& t) {
  if (!t.is_cuda()) value_error("the tensors must be on a CUDA device");
  return t.get_device();
}

// On the call's device, or in pinned host memory (which the device reads).
void same_device(int index, const Tensor& t, const char* name) {
  if (t.is_cuda() ? t.get_device() != index : !t.is_pinned())
    value_error(std::string(name) + " is on " + t.device().str() +
                ", the call's other tensors on cuda:" + std::to_string(index));
}

bool none(PyObject* o) { return o == Py_None; }

int as_int(PyObject* o, const char* name) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    type_error(std::string(name) + " must be an int");
  }
  if (v > 0x7fffffffL || v < -0x7fffffffL - 1)
    value_error(std::string(name) + " does not fit 32 bits");
  return static_cast<int>(v);
}

double as_double(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    type_error(std::string(name) + " must be a number");
  }
  return v;
}

int size32(const Tensor& t, int64_t dim) {
  const int64_t n = t.size(dim);
  if (n > 0x7fffffff) value_error("a dimension does not fit 32 bits");
  return static_cast<int>(n);
}

// The launch block's flag and stream.
int* flag_of(PyObject* o, int index) {
  if (none(o)) return nullptr;
  const Tensor& t = tensor(o, "err_flag");
  if (t.nbytes() < sizeof(int)) value_error("err_flag needs one int32 element");
  same_device(index, t, "err_flag");
  return static_cast<int*>(t.data_ptr());
}

void* stream_of(PyObject* o, int index) {
  if (none(o)) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index)).stream();
  void* p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) {
    PyErr_Clear();
    type_error("stream must be a CUDA stream or its handle");
  }
  return p;
}

// A call on a given stream allocates on it, as one made under that stream would:
// what it frees on its return (a workspace) is not handed to work on another.  What
// it returns is recorded as used on the caller's stream too, so that the caller may
// use it there (having waited for the call's) and drop it.
class OnStream {
  c10::cuda::CUDAGuard device_;
  c10::cuda::CUDAStream caller_;
  std::optional<c10::cuda::CUDAStreamGuard> stream_;

 public:
  OnStream(int index, bool given, void* stream)
      : device_(static_cast<c10::DeviceIndex>(index)),
        caller_(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index))) {
    if (given && caller_.stream() != static_cast<cudaStream_t>(stream))
      stream_.emplace(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(stream),
                                                       static_cast<c10::DeviceIndex>(index)));
  }
  Tensor result(c10::IntArrayRef sizes, const c10::TensorOptions& options) const {
    Tensor t = at::empty(sizes, options);
    if (stream_)
      c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), caller_);
    return t;
  }
};

// The allocations and the library's call run without the interpreter's lock (a
// launch waits when the device's queue is full); it is held again on the way out.
class Unlocked {
  PyThreadState* state_ = PyEval_SaveThread();

 public:
  Unlocked() = default;
  Unlocked(const Unlocked&) = delete;
  ~Unlocked() { PyEval_RestoreThread(state_); }
};

PyObject* status(int st) { return PyLong_FromLong(st); }

void count(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) type_error("wrong number of arguments");
}

// open(path): the library's entry points.
PyObject* open_library(PyObject* const* a, Py_ssize_t n) {
  count(n, 1);
  const char* path = PyUnicode_AsUTF8(a[0]);
  if (!path) return nullptr;
  void* h = dlopen(path, RTLD_NOW | RTLD_LOCAL);
  if (!h) {
    PyErr_SetString(PyExc_RuntimeError, dlerror());
    return nullptr;
  }
#define DECATTN_FIND(name)                                              \
  lib.name = reinterpret_cast<decltype(lib.name)>(dlsym(h, #name));     \
  if (!lib.name) {                                                      \
    PyErr_SetString(PyExc_RuntimeError, "libdecattn has no " #name);    \
    return nullptr;                                                     \
  }
  DECATTN_CALLS(DECATTN_FIND)
#undef DECATTN_FIND
  Py_RETURN_NONE;
}

// paged_plan(cached_lens, new_lens, block_table, free_blocks, free_count,
//   block_size, max_tokens, seq_lens, q_start, slots, positions,
//   free_count_out, err_flag, stream): the five output tensors.
PyObject* paged_plan(PyObject* const* a, Py_ssize_t n) {
  count(n, 14);
  const Tensor& cached = check(a[0], "cached_lens", ScalarType::Int, 1);
  const Tensor& moved = check(a[1], "new_lens", ScalarType::Int, 1);
  const Tensor& table = check(a[2], "block_table", ScalarType::Int, 2);
  const Tensor& free = check(a[3], "free_blocks", ScalarType::Int, 1);
  const Tensor& top = check(a[4], "free_count", ScalarType::Int, 1);
  const int B = size32(cached, 0), tokens = as_int(a[6], "max_tokens");
  if (moved.size(0) != B || table.size(0) != B || top.size(0) != 1)
    value_error("paged_plan: shape mismatch");
  if (tokens < 0) value_error("max_tokens must not be negative");
  const int index = cuda_index(cached);
  same_device(index, moved, "new_lens");
  same_device(index, table, "block_table");
  same_device(index, free, "free_blocks");
  same_device(index, top, "free_count");
  decattn_launch L = {};
  L.batch = B;
  L.num_blocks = size32(free, 0);
  L.block_size = as_int(a[5], "block_size");
  L.max_blocks_per_seq = size32(table, 1);
  L.err_flag = flag_of(a[12], index);
  L.stream = stream_of(a[13], index);
  const char* names[] = {"seq_lens", "q_start", "slots", "positions", "free_count_out"};
  const int64_t sizes[] = {B, static_cast<int64_t>(B) + 1, tokens, tokens, 1};
  Tensor out[5];
  for (int k = 0; k < 5; ++k) {
    if (!none(a[7 + k])) {
      out[k] = check(a[7 + k], names[k], ScalarType::Int, 1);
      if (out[k].size(0) != sizes[k])
        value_error(std::string(names[k]) + ": expected [" + std::to_string(sizes[k]) +
                    "], got shape " + shape_of(out[k]));
      same_device(index, out[k], names[k]);
    }
  }
  auto at_ = [](const Tensor& t) { return t.data_ptr<int>(); };
  const bool given = !none(a[13]);
  const int st = [&] {
    const Unlocked unlocked;
    const OnStream guard(index, given, L.stream);
    // One allocation for the outputs that were not given (a call of at::empty
    // takes 0.6 us, the smallest step's kernel 4).
    int64_t total = 0;
    for (int k = 0; k < 5; ++k)
      if (!out[k].defined()) total += (sizes[k] + 63) / 64 * 64;
    if (total) {
      const Tensor slab = guard.result({total}, cached.options());
      int64_t at = 0;
      for (int k = 0; k < 5; ++k) {
        if (out[k].defined()) continue;
        out[k] = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(slab.storage()),
                                                          slab.key_set(), slab.dtype());
        out[k].unsafeGetTensorImpl()->set_sizes_and_strides(
            c10::IntArrayRef{sizes[k]}, c10::IntArrayRef{1}, at);
        at += (sizes[k] + 63) / 64 * 64;
      }
    }
    return lib.paged_plan(at_(cached), at_(moved), at_(table), at_(free), at_(top), at_(out[4]),
                          at_(out[0]), at_(out[1]), at_(out[2]), at_(out[3]), tokens, &L);
  }();
  if (st != DECATTN_OK) return status(st);
  PyObject* r = PyTuple_New(5);
  for (int k = 0; r && k < 5; ++k) PyTuple_SET_ITEM(r, k, THPVariable_Wrap(out[k]));
  return r;
}

// A [tokens, heads, 128] tensor whose heads are contiguous within a token (a
// part of a wider projection's output will do): its token stride.
int64_t packed_rows(const Tensor& t, const char* name) {
  if (t.dim() != 3)
    value_error(std::string(name) + ": expected 3 dims, got shape " + shape_of(t));
  const int64_t T = t.size(0), h = t.size(1), d = t.size(2);
  if (t.numel() && ((d > 1 && t.stride(2) != 1) || (h > 1 && t.stride(1) != d)))
    value_error(std::string(name) + ": a token's heads must be contiguous");
  return T > 1 ? t.stride(0) : h * d;
}

const float* scale_of(PyObject* o, const char* name, int64_t heads, int index) {
  const Tensor& t = check(o, name, ScalarType::Float, 1);
  if (t.size(0) != heads) value_error(std::string(name) + " must be [h_kv]");
  same_device(index, t, name);
  return t.data_ptr<float>();
}

// rope_append(q, k_new, v_new, k_scale, v_scale, positions, rope's address, its
//   number of axes, slots, k_cache, v_cache, q_out, err_flag, stream): q_out.
//   k_scale None: a 16-bit cache.
PyObject* rope_append(PyObject* const* a, Py_ssize_t n) {
  count(n, 14);
  const bool fp8 = !none(a[3]);
  const Tensor& q = tensor(a[0], "q");
  const int64_t qs = packed_rows(q, "q");
  const int dtype = dtype16(q, "q");
  const Tensor &k = tensor(a[1], "k_new"), &v = tensor(a[2], "v_new");
  for (const Tensor* t : {&k, &v})
    if (t->scalar_type() != q.scalar_type())
      type_error(std::string(t == &k ? "k_new" : "v_new") + ": expected " +
                 name_of(q.scalar_type()) + ", got " + name_of(t->scalar_type()));
  const int64_t ks = packed_rows(k, "k_new"), vs = packed_rows(v, "v_new");
  const Tensor& pos = check(a[5], "positions", ScalarType::Int, -1);
  const Tensor& slots = check(a[8], "slots", ScalarType::Int, 1);
  const Tensor& kc = fp8 ? check_codes(a[9], "k_codes") : check(a[9], "k_cache", q.scalar_type(), 4);
  const Tensor& vc =
      fp8 ? check_codes(a[10], "v_codes") : check(a[10], "v_cache", q.scalar_type(), 4);
  const int T = size32(q, 0), h_q = size32(q, 1), d = size32(q, 2), h_kv = size32(k, 1);
  if (k.size(0) != T || k.size(2) != d || v.sizes() != k.sizes() || kc.size(2) != h_kv ||
      kc.size(3) != d || vc.sizes() != kc.sizes() || slots.size(0) != T)
    value_error("rope_append: shape mismatch");
  const int axes = as_int(a[7], "n_axes");
  if (!(pos.dim() == 2 && pos.size(0) == axes && pos.size(1) == T) &&
      !(axes == 1 && pos.dim() == 1 && pos.size(0) == T))
    value_error("positions must be [" + std::to_string(axes) + ", " + std::to_string(T) + "]");
  const int index = cuda_index(q);
  const float *sk = nullptr, *sv = nullptr;
  if (fp8) {
    sk = scale_of(a[3], "k_scale", h_kv, index);
    sv = scale_of(a[4], "v_scale", h_kv, index);
  }
  same_device(index, k, "k_new");
  same_device(index, v, "v_new");
  same_device(index, pos, "positions");
  same_device(index, slots, "slots");
  same_device(index, kc, "k_cache");
  same_device(index, vc, "v_cache");
  decattn_launch L = {};
  L.batch = 1;
  L.num_blocks = size32(kc, 0);
  L.block_size = size32(kc, 1);
  L.dtype = dtype;
  L.err_flag = flag_of(a[12], index);
  L.stream = stream_of(a[13], index);
  const auto* rope = static_cast<const decattn_rope*>(PyLong_AsVoidPtr(a[6]));
  Tensor out;
  if (!none(a[11])) {
    out = check(a[11], "q_out", q.scalar_type(), 3);
    if (out.sizes() != q.sizes())
      value_error("q_out: expected shape " + shape_of(q) + ", got " + shape_of(out));
    same_device(index, out, "q_out");
  }
  const void *qp = q.data_ptr(), *kp = k.data_ptr(), *vp = v.data_ptr();
  void *kcp = kc.data_ptr(), *vcp = vc.data_ptr();
  const int *pp = pos.data_ptr<int>(), *sp = slots.data_ptr<int>();
  const bool given = !none(a[13]);
  const int st = [&] {
    const Unlocked unlocked;
    const OnStream guard(index, given, L.stream);
    if (!out.defined()) out = guard.result({T, h_q, d}, q.options());
    return fp8 ? lib.gqa_rope_append_fp8kv(qp, kp, vp, qs, ks, vs, sk, sv, pp, rope, sp,
                                           out.data_ptr(), kcp, vcp, T, h_q, h_kv, d, &L)
               : lib.gqa_rope_append(qp, kp, vp, qs, ks, vs, pp, rope, sp, out.data_ptr(), kcp,
                                     vcp, T, h_q, h_kv, d, &L);
  }();
  return st != DECATTN_OK ? status(st) : THPVariable_Wrap(out);
}

// q, the caches, the scales and the table of decode and prefill.
struct Attention {
  const Tensor *q, *kc, *vc, *table, *lens;
  const float *sk = nullptr, *sv = nullptr;
  int dtype, h_q, h_kv, d, index;
  bool fp8;
  // q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens.  `decode`: a row of
  // q for each sequence, so that the table and the lengths must reach as far.
  Attention(PyObject* const* a, bool decode) : fp8(!none(a[3])) {
    const Tensor& t = tensor(a[0], "q");
    q = &check(a[0], "q", t.scalar_type(), 3);
    dtype = dtype16(t, "q");
    kc = fp8 ? &check_codes(a[1], "k_codes") : &check(a[1], "k_cache", t.scalar_type(), 4);
    vc = fp8 ? &check_codes(a[2], "v_codes") : &check(a[2], "v_cache", t.scalar_type(), 4);
    table = &check(a[5], "block_table", ScalarType::Int, 2);
    lens = &check(a[6], "seq_lens", ScalarType::Int, 1);
    h_q = size32(t, 1);
    d = size32(t, 2);
    h_kv = size32(*kc, 2);
    if (kc->size(3) != d || vc->sizes() != kc->sizes())
      value_error(fp8 ? "k_codes / v_codes shape mismatch" : "k_cache / v_cache shape mismatch");
    if (decode && (table->size(0) < t.size(0) || lens->size(0) < t.size(0)))
      value_error("block_table and seq_lens need an entry for each of the " +
                  std::to_string(t.size(0)) + " rows of q, got " + std::to_string(table->size(0)) +
                  " and " + std::to_string(lens->size(0)));
    if (h_kv < 1 || h_q % h_kv != 0)
      value_error("h_q=" + std::to_string(h_q) + " is not a multiple of h_kv=" +
                  std::to_string(h_kv));
    index = cuda_index(t);
    if (fp8) {
      sk = scale_of(a[3], "k_scale", h_kv, index);
      sv = scale_of(a[4], "v_scale", h_kv, index);
    }
    same_device(index, *kc, "k_cache");
    same_device(index, *vc, "v_cache");
    same_device(index, *table, "block_table");
    same_device(index, *lens, "seq_lens");
  }
  decattn_launch launch(int batch, int max_seq_len, PyObject* flag, PyObject* stream) const {
    decattn_launch L = {};
    L.batch = batch;
    L.num_blocks = size32(*kc, 0);
    L.block_size = size32(*kc, 1);
    L.max_blocks_per_seq = size32(*table, 1);
    L.max_seq_len = max_seq_len;
    L.dtype = dtype;
    L.err_flag = flag_of(flag, index);
    L.stream = stream_of(stream, index);
    return L;
  }
  // The given output (undefined: none).  `exact`: [tokens, h_q, d]; else any
  // contiguous tensor with room for it.
  Tensor output(PyObject* o, bool exact) const {
    if (none(o)) return Tensor();
    const Tensor& t = check(o, "out", q->scalar_type(), exact ? 3 : -1);
    if (exact ? t.sizes() != q->sizes() : t.numel() < q->numel())
      value_error("out: expected shape " + shape_of(*q) + ", got " + shape_of(t));
    same_device(index, t, "out");
    return t;
  }
  // The given workspace (undefined: none).
  Tensor workspace(PyObject* o) const {
    if (none(o)) return Tensor();
    const Tensor& t = tensor(o, "workspace");
    // (Bytes alone count: any order of strides will do, but none of them may lie
    // between the tensor's elements.)
    if (!t.is_non_overlapping_and_dense()) value_error("workspace must be dense");
    same_device(index, t, "workspace");
    return t;
  }
  // What was not given is allocated: the output, `need` bytes of workspace.
  void* allocate(const OnStream& guard, Tensor& out, Tensor& ws, size_t need,
                 decattn_launch& L) const {
    if (!out.defined()) out = guard.result(q->sizes(), q->options());
    if (!ws.defined() && need)
      ws = at::empty({static_cast<int64_t>(need)}, q->options().dtype(ScalarType::Byte));
    if (ws.defined()) {
      L.workspace = ws.data_ptr();
      L.workspace_bytes = ws.nbytes();
    }
    return out.data_ptr();
  }
};

// decode(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, scale,
//   max_seq_len, window or None, sinks, num_splits, out, workspace, err_flag,
//   stream): out.
PyObject* decode(PyObject* const* a, Py_ssize_t n) {
  count(n, 16);
  const Attention x(a, true);
  const float scale = static_cast<float>(as_double(a[7], "scale"));
  const int max_len = as_int(a[8], "max_seq_len"), sinks = as_int(a[10], "sinks");
  const bool windowed = !none(a[9]);
  const int window = windowed ? as_int(a[9], "window") : 0;
  const int B = size32(*x.q, 0);
  decattn_launch L = x.launch(B, max_len, a[14], a[15]);
  L.num_splits = as_int(a[11], "num_splits");
  Tensor out = x.output(a[12], false), ws = x.workspace(a[13]);
  const void *q = x.q->data_ptr(), *kc = x.kc->data_ptr(), *vc = x.vc->data_ptr();
  const int *bt = x.table->data_ptr<int>(), *sl = x.lens->data_ptr<int>();
  const bool given = !none(a[15]);
  const int st = [&] {
    const Unlocked unlocked;
    const OnStream guard(x.index, given, L.stream);
    if (L.num_splits == 0) {
      const int ns =
          windowed ? lib.gqa_decode_sinks_plan_splits(B, x.h_q, x.h_kv, x.d, max_len, window,
                                                      sinks, L.block_size, x.fp8 ? 1 : 2, 0)
          : x.fp8  ? lib.gqa_decode_fp8kv_plan_splits(B, x.h_q, x.h_kv, x.d, max_len, 0)
                   : lib.gqa_decode_plan_splits(B, x.h_q, x.h_kv, x.d, max_len, 0);
      if (ns < 0) return ns;
      L.num_splits = ns;
    }
    const int ns = L.num_splits;
    void* o = x.allocate(guard, out, ws,
                         ns > 1 ? lib.gqa_decode_workspace_size(B, x.h_q, x.d, ns) : 0, L);
    if (!windowed)
      return x.fp8 ? lib.gqa_decode_fp8kv(q, kc, vc, x.sk, x.sv, bt, sl, o, x.h_q, x.h_kv, x.d,
                                          scale, &L)
                   : lib.gqa_decode(q, kc, vc, bt, sl, o, x.h_q, x.h_kv, x.d, scale, &L);
    if (sinks == 0)
      return x.fp8 ? lib.gqa_decode_fp8kv_window(q, kc, vc, x.sk, x.sv, bt, sl, o, x.h_q, x.h_kv,
                                                 x.d, scale, window, &L)
                   : lib.gqa_decode_window(q, kc, vc, bt, sl, o, x.h_q, x.h_kv, x.d, scale,
                                           window, &L);
    return x.fp8 ? lib.gqa_decode_fp8kv_sinks(q, kc, vc, x.sk, x.sv, bt, sl, o, x.h_q, x.h_kv, x.d,
                                              scale, window, sinks, &L)
                 : lib.gqa_decode_sinks(q, kc, vc, bt, sl, o, x.h_q, x.h_kv, x.d, scale, window,
                                        sinks, &L);
  }();
  return st != DECATTN_OK ? status(st) : THPVariable_Wrap(out);
}

// decode_blocks(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens,
//   selected, scale, max_seq_len, num_splits, out, workspace, err_flag, stream): out.
PyObject* decode_blocks(PyObject* const* a, Py_ssize_t n) {
  count(n, 15);
  const Attention x(a, true);
  const Tensor& selected = check(a[7], "selected", ScalarType::Int, 3);
  const int B = size32(*x.q, 0), most = size32(selected, 2);
  if (selected.size(0) < B || selected.size(1) != x.h_kv)
    value_error("selected must be [" + std::to_string(B) + ", " + std::to_string(x.h_kv) +
                ", count], got shape " + shape_of(selected));
  same_device(x.index, selected, "selected");
  const float scale = static_cast<float>(as_double(a[8], "scale"));
  const int max_len = as_int(a[9], "max_seq_len");
  decattn_launch L = x.launch(B, max_len, a[13], a[14]);
  L.num_splits = as_int(a[10], "num_splits");
  Tensor out = x.output(a[11], false), ws = x.workspace(a[12]);
  const void *q = x.q->data_ptr(), *kc = x.kc->data_ptr(), *vc = x.vc->data_ptr();
  const int *bt = x.table->data_ptr<int>(), *sl = x.lens->data_ptr<int>();
  const int* some = selected.data_ptr<int>();
  const bool given = !none(a[14]);
  const int st = [&] {
    const Unlocked unlocked;
    const OnStream guard(x.index, given, L.stream);
    if (L.num_splits == 0) {
      const int ns = lib.gqa_decode_blocks_plan_splits(B, x.h_q, x.h_kv, x.d, max_len, most,
                                                       L.block_size, x.fp8 ? 1 : 2, 0);
      if (ns < 0) return ns;
      L.num_splits = ns;
    }
    const int ns = L.num_splits;
    void* o = x.allocate(guard, out, ws,
                         ns > 1 ? lib.gqa_decode_workspace_size(B, x.h_q, x.d, ns) : 0, L);
    return x.fp8 ? lib.gqa_decode_fp8kv_blocks(q, kc, vc, x.sk, x.sv, bt, sl, some, o, x.h_q,
                                               x.h_kv, x.d, scale, most, &L)
                 : lib.gqa_decode_blocks(q, kc, vc, bt, sl, some, o, x.h_q, x.h_kv, x.d, scale,
                                         most, &L);
  }();
  return st != DECATTN_OK ? status(st) : THPVariable_Wrap(out);
}

// A cache's weights: float32 [num_blocks, h_kv, block_size].
const Tensor& check_weights(PyObject* o, const Tensor& cache, int index) {
  const Tensor& t = check(o, "weights", ScalarType::Float, 3);
  if (t.size(0) != cache.size(0) || t.size(1) != cache.size(2) || t.size(2) != cache.size(1))
    value_error("weights must be [num_blocks, h_kv, block_size], got shape " + shape_of(t));
  same_device(index, t, "weights");
  return t;
}

// decode_weights(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens,
//   weights, weighed_lens or None, scale, decay, max_seq_len, num_splits, out,
//   workspace, err_flag, stream): out.
PyObject* decode_weights(PyObject* const* a, Py_ssize_t n) {
  count(n, 17);
  const Attention x(a, true);
  const Tensor& weights = check_weights(a[7], *x.kc, x.index);
  const int B = size32(*x.q, 0);
  const int* weighed = nullptr;
  if (!none(a[8])) {
    const Tensor& t = check(a[8], "weighed_lens", ScalarType::Int, 1);
    if (t.size(0) < B) value_error("weighed_lens needs an entry for each row of q");
    same_device(x.index, t, "weighed_lens");
    weighed = t.data_ptr<int>();
  }
  const float scale = static_cast<float>(as_double(a[9], "scale"));
  const float decay = static_cast<float>(as_double(a[10], "decay"));
  const int max_len = as_int(a[11], "max_seq_len");
  decattn_launch L = x.launch(B, max_len, a[15], a[16]);
  L.num_splits = as_int(a[12], "num_splits");
  Tensor out = x.output(a[13], false), ws = x.workspace(a[14]);
  const void *q = x.q->data_ptr(), *kc = x.kc->data_ptr(), *vc = x.vc->data_ptr();
  const int *bt = x.table->data_ptr<int>(), *sl = x.lens->data_ptr<int>();
  float* w = weights.data_ptr<float>();
  const bool given = !none(a[16]);
  const int st = [&] {
    const Unlocked unlocked;
    const OnStream guard(x.index, given, L.stream);
    if (L.num_splits == 0) {
      const int ns = lib.gqa_decode_weights_plan_splits(B, x.h_q, x.h_kv, x.d, max_len,
                                                        x.fp8 ? 1 : 2, 0);
      if (ns < 0) return ns;
      L.num_splits = ns;
    }
    void* o = x.allocate(
        guard, out, ws,
        lib.gqa_decode_weights_workspace_size(B, x.h_q, x.d, max_len, L.num_splits), L);
    return x.fp8 ? lib.gqa_decode_fp8kv_weights(q, kc, vc, x.sk, x.sv, bt, sl, weighed, w, o,
                                                x.h_q, x.h_kv, x.d, scale, decay, &L)
                 : lib.gqa_decode_weights(q, kc, vc, bt, sl, weighed, w, o, x.h_q, x.h_kv, x.d,
                                          scale, decay, &L);
  }();
  return st != DECATTN_OK ? status(st) : THPVariable_Wrap(out);
}

// A cache (or its bounds) of any of the library's types, and how it is numbered.
struct Kind {
  int bytes, dtype;
};
Kind kind_of(const Tensor& t, const char* name) {
  switch (t.scalar_type()) {
    case ScalarType::Half: return {2, DECATTN_FP16};
    case ScalarType::BFloat16: return {2, DECATTN_BF16};
    case ScalarType::Byte:
    case ScalarType::Float8_e4m3fn: return {1, DECATTN_BF16};
    default:
      type_error(std::string(name) + " must be float16, bfloat16, float8_e4m3fn or uint8");
  }
}

// block_table [B, max_blocks] and seq_lens [B] of a call without a query.
void check_lists(const Tensor& table, const Tensor& lens, int index) {
  if (table.size(0) != lens.size(0))
    value_error("block_table must have a row for each of the " + std::to_string(lens.size(0)) +
                " sequences, got " + std::to_string(table.size(0)));
  same_device(index, table, "block_table");
  same_device(index, lens, "seq_lens");
}

// block_bounds(k_cache, block_table, seq_lens, bounds, first_lens or None,
//   max_seq_len, err_flag, stream): bounds.
PyObject* block_bounds(PyObject* const* a, Py_ssize_t n) {
  count(n, 8);
  const Tensor& k = tensor(a[0], "k_cache");
  const Kind kind = kind_of(k, "k_cache");
  check(a[0], "k_cache", k.scalar_type(), 4);
  const Tensor& table = check(a[1], "block_table", ScalarType::Int, 2);
  const Tensor& lens = check(a[2], "seq_lens", ScalarType::Int, 1);
  const Tensor& bounds = tensor(a[3], "bounds");
  if (kind_of(bounds, "bounds").bytes != kind.bytes ||
      (kind.bytes == 2 && bounds.scalar_type() != k.scalar_type()))
    type_error("bounds must be of k_cache's type");
  check(a[3], "bounds", bounds.scalar_type(), 4);
  if (bounds.size(0) != k.size(0) || bounds.size(1) != 2 || bounds.size(2) != k.size(2) ||
      bounds.size(3) != k.size(3))
    value_error("bounds must be [num_blocks, 2, h_kv, d], got shape " + shape_of(bounds));
  const int index = cuda_index(k);
  check_lists(table, lens, index);
  same_device(index, bounds, "bounds");
  const int* first = nullptr;
  if (!none(a[4])) {
    const Tensor& t = check(a[4], "first_lens", ScalarType::Int, 1);
    if (t.size(0) != lens.size(0)) value_error("first_lens must have seq_lens' shape");
    same_device(index, t, "first_lens");
    first = t.data_ptr<int>();
  }
  decattn_launch L = {};
  L.batch = size32(lens, 0);
  L.num_blocks = size32(k, 0);
  L.block_size = size32(k, 1);
  L.max_blocks_per_seq = size32(table, 1);
  L.max_seq_len = as_int(a[5], "max_seq_len");
  L.dtype = kind.dtype;
  L.err_flag = flag_of(a[6], index);
  L.stream = stream_of(a[7], index);
  const bool given = !none(a[7]);
  const int h_kv = size32(k, 2), d = size32(k, 3);
  const void* kp = k.data_ptr();
  void* bp = bounds.data_ptr();
  const int *bt = table.data_ptr<int>(), *sl = lens.data_ptr<int>();
  const int st = [&] {
    const Unlocked unlocked;
    const OnStream guard(index, given, L.stream);
    return lib.gqa_block_bounds(kp, bt, first, sl, bp, h_kv, d, kind.bytes, &L);
  }();
  return st != DECATTN_OK ? status(st) : THPVariable_Wrap(bounds);
}

// select_blocks(q, bounds, block_table, seq_lens, block_size, max_seq_len,
//   count, first, last, out, workspace, err_flag, stream): selected.
PyObject* select_blocks(PyObject* const* a, Py_ssize_t n) {
  count(n, 13);
  const Tensor& q = tensor(a[0], "q");
  const int dtype = dtype16(q, "q");
  check(a[0], "q", q.scalar_type(), 3);
  const Tensor& bounds = tensor(a[1], "bounds");
  const Kind kind = kind_of(bounds, "bounds");
  check(a[1], "bounds", kind.bytes == 2 ? q.scalar_type() : bounds.scalar_type(), 4);
  const Tensor& table = check(a[2], "block_table", ScalarType::Int, 2);
  const Tensor& lens = check(a[3], "seq_lens", ScalarType::Int, 1);
  const int B = size32(q, 0), h_q = size32(q, 1), d = size32(q, 2), h_kv = size32(bounds, 2);
  if (bounds.size(1) != 2 || bounds.size(3) != d)
    value_error("bounds must be [num_blocks, 2, h_kv, d], got shape " + shape_of(bounds));
  if (table.size(0) < B || lens.size(0) < B)
    value_error("block_table and seq_lens need an entry for each of the " + std::to_string(B) +
                " rows of q, got " + std::to_string(table.size(0)) + " and " +
                std::to_string(lens.size(0)));
  if (h_kv < 1 || h_q % h_kv != 0)
    value_error("h_q=" + std::to_string(h_q) + " is not a multiple of h_kv=" + std::to_string(h_kv));
  const int index = cuda_index(q);
  same_device(index, bounds, "bounds");
  same_device(index, table, "block_table");
  same_device(index, lens, "seq_lens");
  decattn_launch L = {};
  L.batch = B;
  L.num_blocks = size32(bounds, 0);
  L.block_size = as_int(a[4], "block_size");
  L.max_blocks_per_seq = size32(table, 1);
  L.max_seq_len = as_int(a[5], "max_seq_len");
  L.dtype = dtype;
  L.err_flag = flag_of(a[11], index);
  L.stream = stream_of(a[12], index);
  const int most = as_int(a[6], "count"), first = as_int(a[7], "first"),
            last = as_int(a[8], "last");
  if (most < 1) value_error("count must be at least 1");
  Tensor out, ws;
  if (!none(a[9])) {
    out = check(a[9], "out", ScalarType::Int, 3);
    if (out.size(0) != B || out.size(1) != h_kv || out.size(2) != most)
      value_error("out must be [" + std::to_string(B) + ", " + std::to_string(h_kv) + ", " +
                  std::to_string(most) + "], got shape " + shape_of(out));
    same_device(index, out, "out");
  }
  if (!none(a[10])) {
    ws = tensor(a[10], "workspace");
    if (!ws.is_non_overlapping_and_dense()) value_error("workspace must be dense");
    same_device(index, ws, "workspace");
  }
  const bool given = !none(a[12]);
  const void *qp = q.data_ptr(), *bp = bounds.data_ptr();
  const int *bt = table.data_ptr<int>(), *sl = lens.data_ptr<int>();
  const int st = [&] {
    const Unlocked unlocked;
    const OnStream guard(index, given, L.stream);
    if (!out.defined())
      out = guard.result({B, h_kv, most}, q.options().dtype(ScalarType::Int));
    const size_t need =
        lib.gqa_select_workspace_size(B, h_kv, L.max_seq_len, L.block_size, most);
    if (!ws.defined() && need)
      ws = at::empty({static_cast<int64_t>(need)}, q.options().dtype(ScalarType::Byte));
    if (ws.defined()) {
      L.workspace = ws.data_ptr();
      L.workspace_bytes = ws.nbytes();
    }
    return lib.gqa_select_blocks(qp, bp, bt, sl, out.data_ptr<int>(), h_q, h_kv, d, kind.bytes,
                                 most, first, last, &L);
  }();
  return st != DECATTN_OK ? status(st) : THPVariable_Wrap(out);
}

// kv_evict(k_cache, v_cache, weights, block_table, seq_lens, max_seq_len, keep,
//   recent, limit, new_lens, kept, err_flag, stream): (new_lens, kept).
PyObject* kv_evict(PyObject* const* a, Py_ssize_t n) {
  count(n, 13);
  const Tensor& k = tensor(a[0], "k_cache");
  const Kind kind = kind_of(k, "k_cache");
  check(a[0], "k_cache", k.scalar_type(), 4);
  const Tensor& v = check(a[1], "v_cache", k.scalar_type(), 4);
  if (v.sizes() != k.sizes()) value_error("k_cache / v_cache shape mismatch");
  const int index = cuda_index(k);
  same_device(index, v, "v_cache");
  const Tensor& weights = check_weights(a[2], k, index);
  const Tensor& table = check(a[3], "block_table", ScalarType::Int, 2);
  const Tensor& lens = check(a[4], "seq_lens", ScalarType::Int, 1);
  check_lists(table, lens, index);
  decattn_launch L = {};
  const int B = L.batch = size32(lens, 0);
  L.num_blocks = size32(k, 0);
  L.block_size = size32(k, 1);
  L.max_blocks_per_seq = size32(table, 1);
  L.max_seq_len = as_int(a[5], "max_seq_len");
  L.dtype = kind.dtype;
  L.err_flag = flag_of(a[11], index);
  L.stream = stream_of(a[12], index);
  const int keep = as_int(a[6], "keep"), recent = as_int(a[7], "recent"),
            limit = as_int(a[8], "limit"), h_kv = size32(k, 2), d = size32(k, 3);
  if (keep < 1) value_error("keep must be at least 1");
  Tensor moved, kept;
  if (!none(a[9])) {
    moved = check(a[9], "new_lens", ScalarType::Int, 1);
    if (moved.size(0) != B) value_error("new_lens must be [" + std::to_string(B) + "]");
    same_device(index, moved, "new_lens");
  }
  if (!none(a[10])) {
    kept = check(a[10], "kept", ScalarType::Int, 3);
    if (kept.size(0) != B || kept.size(1) != h_kv || kept.size(2) != keep)
      value_error("kept must be [" + std::to_string(B) + ", " + std::to_string(h_kv) + ", " +
                  std::to_string(keep) + "], got shape " + shape_of(kept));
    same_device(index, kept, "kept");
  }
  const bool given = !none(a[12]);
  void *kp = k.data_ptr(), *vp = v.data_ptr();
  float* w = weights.data_ptr<float>();
  const int *bt = table.data_ptr<int>(), *sl = lens.data_ptr<int>();
  const int st = [&] {
    const Unlocked unlocked;
    const OnStream guard(index, given, L.stream);
    const at::TensorOptions i32 = weights.options().dtype(ScalarType::Int);
    if (!moved.defined()) moved = guard.result({B}, i32);
    if (!kept.defined()) kept = guard.result({B, h_kv, keep}, i32);
    return lib.gqa_kv_evict(kp, vp, w, bt, sl, moved.data_ptr<int>(), kept.data_ptr<int>(), h_kv,
                            d, kind.bytes, keep, recent, limit, &L);
  }();
  if (st != DECATTN_OK) return status(st);
  PyObject* r = PyTuple_New(2);
  if (r) {
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(moved));
    PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(kept));
  }
  return r;
}

// prefill(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, q_start,
//   scale, max_q_len, max_seq_len, window (0: none), sinks, num_splits, out,
//   workspace, err_flag, stream): out.
PyObject* prefill(PyObject* const* a, Py_ssize_t n) {
  count(n, 18);
  const Attention x(a, false);
  const Tensor& start = check(a[7], "q_start", ScalarType::Int, 1);
  const int B = size32(*x.lens, 0), T = size32(*x.q, 0);
  if (x.table->size(0) != B || start.size(0) != B + 1)
    value_error("block_table must be [B, max_blocks] and q_start [B + 1]");
  same_device(x.index, start, "q_start");
  const float scale = static_cast<float>(as_double(a[8], "scale"));
  const int max_q = as_int(a[9], "max_q_len"), max_len = as_int(a[10], "max_seq_len");
  const int window = as_int(a[11], "window"), sinks = as_int(a[12], "sinks");
  decattn_launch L = x.launch(B, max_len, a[16], a[17]);
  L.num_splits = as_int(a[13], "num_splits");
  Tensor out = x.output(a[14], true), ws = x.workspace(a[15]);
  const void *q = x.q->data_ptr(), *kc = x.kc->data_ptr(), *vc = x.vc->data_ptr();
  const int *bt = x.table->data_ptr<int>(), *sl = x.lens->data_ptr<int>();
  const int* qs = start.data_ptr<int>();
  const bool given = !none(a[17]);
  const int st = [&] {
    const Unlocked unlocked;
    const OnStream guard(x.index, given, L.stream);
    if (L.num_splits == 0) {
      const int ns = lib.gqa_prefill_plan_splits(B, T, max_q, x.h_q, x.h_kv, x.d, max_len, window,
                                                 sinks, 0);
      if (ns < 0) return ns;
      L.num_splits = ns;
    }
    const int ns = L.num_splits;
    void* o = x.allocate(
        guard, out, ws, T && ns > 1 ? lib.gqa_prefill_workspace_size(T, x.h_q, x.d, ns) : 0, L);
    return x.fp8 ? lib.gqa_prefill_fp8kv(q, kc, vc, x.sk, x.sv, bt, qs, sl, o, T, max_q, x.h_q,
                                         x.h_kv, x.d, scale, window, sinks, &L)
                 : lib.gqa_prefill(q, kc, vc, bt, qs, sl, o, T, max_q, x.h_q, x.h_kv, x.d, scale,
                                   window, sinks, &L);
  }();
  return st != DECATTN_OK ? status(st) : THPVariable_Wrap(out);
}

// Refusals and C++ exceptions (an allocation that fails) become Python's.
template <PyObject* (*kCall)(PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    return kCall(args, n);
  } catch (const Refused& r) {
    PyErr_SetString(r.type, r.what.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*kCall)(PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name,
          reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(&guarded<kCall>)),
          METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<open_library>("open"), method<paged_plan>("paged_plan"),
                         method<rope_append>("rope_append"), method<decode>("decode"),
                         method<prefill>("prefill"), method<decode_blocks>("decode_blocks"),
                         method<decode_weights>("decode_weights"),
                         method<block_bounds>("block_bounds"),
                         method<select_blocks>("select_blocks"),
                         method<kv_evict>("kv_evict"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
