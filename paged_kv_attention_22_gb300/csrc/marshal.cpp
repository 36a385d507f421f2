// Argument marshalling of the Python binding for the calls on 4-bit caches and
// of eviction: checks torch tensors (type, dtype, shape, device, layout), takes
// their pointers and the current CUDA stream, and calls the C entries of
// include/pkv.h. It computes nothing; a call costs about a microsecond here
// where checks in Python cost ten to twenty, several times the launch itself.
//
// Every function takes its arguments by position and returns the pkv_status as
// an int (some with the tensors that they allocated); the functions of the
// package raise on it. `None` stands for an optional tensor left out.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <exception>

#include "pkv.h"

namespace {

// Raised (and translated at the module's boundary) once a Python error is set.
struct PythonError {};

[[noreturn]] void fail(PyObject *type, const char *format, const char *a = "", const char *b = "") {
  PyErr_Format(type, format, a, b);
  throw PythonError{};
}

// The arguments of one call, in order.
class Args {
 public:
  Args(const char *function, PyObject *const *args, Py_ssize_t n, Py_ssize_t want) : args_(args) {
    if (n != want) fail(PyExc_TypeError, "%s: wrong number of arguments", function);
  }

  // A contiguous CUDA tensor of this dtype and number of dimensions on the
  // current device.
  const at::Tensor &tensor(const char *name, at::ScalarType dtype, int64_t ndim) {
    return check(next(), name, dtype, ndim);
  }
  // The same, or nullptr for None.
  const at::Tensor *maybe(const char *name, at::ScalarType dtype, int64_t ndim) {
    PyObject *o = next();
    return o == Py_None ? nullptr : &check(o, name, dtype, ndim);
  }
  // A (codes, params) pair.
  void cache(const char *name, const at::Tensor **codes, const at::Tensor **params) {
    PyObject *o = next();
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 2)
      fail(PyExc_TypeError, "%s must be a Q4Cache or a (codes, params) pair", name);
    *codes = &check(PyTuple_GET_ITEM(o, 0), name, at::kByte, 4);
    *params = &check(PyTuple_GET_ITEM(o, 1), name, at::kBFloat16, 5);
  }
  int32_t i32(const char *name) {
    const long long v = PyLong_AsLongLong(next());
    if (v == -1 && PyErr_Occurred()) throw PythonError{};
    if (v < INT32_MIN || v > INT32_MAX) fail(PyExc_ValueError, "%s does not fit in 32 bits", name);
    return static_cast<int32_t>(v);
  }
  float f32() {
    const double v = PyFloat_AsDouble(next());
    if (v == -1.0 && PyErr_Occurred()) throw PythonError{};
    return static_cast<float>(v);
  }
  // A torch.cuda.Stream, or None for the current stream.
  void *stream() {
    PyObject *o = next();
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
    PyObject *handle = PyObject_GetAttrString(o, "cuda_stream");
    if (handle == nullptr) throw PythonError{};
    void *p = PyLong_AsVoidPtr(handle);
    Py_DECREF(handle);
    if (p == nullptr && PyErr_Occurred()) throw PythonError{};
    return p;
  }

 private:
  PyObject *next() { return args_[at_++]; }

  const at::Tensor &check(PyObject *o, const char *name, at::ScalarType dtype, int64_t ndim) {
    if (!THPVariable_Check(o)) fail(PyExc_TypeError, "%s must be a torch.Tensor", name);
    const at::Tensor &t = THPVariable_Unpack(o);
    if (t.scalar_type() != dtype) fail(PyExc_TypeError, "%s must be %s", name, c10::toString(dtype));
    if (t.dim() != ndim) fail(PyExc_ValueError, "%s has the wrong number of dims", name);
    if (!t.is_cuda()) fail(PyExc_ValueError, "%s must be a CUDA tensor", name);
    if (!t.is_contiguous()) fail(PyExc_ValueError, "%s must be contiguous", name);
    if (device_ < 0) device_ = c10::cuda::current_device();
    if (t.get_device() != device_) fail(PyExc_ValueError, "%s is not on the current device", name);
    return t;
  }

  PyObject *const *args_;
  Py_ssize_t at_ = 0;
  int device_ = -1;
};

void require(bool ok) {
  if (!ok) fail(PyExc_ValueError, "inconsistent shapes");
}

int32_t size32(const at::Tensor &t, int64_t dim) {
  const int64_t n = t.size(dim);
  if (n > INT32_MAX) fail(PyExc_ValueError, "a dimension does not fit in 32 bits");
  return static_cast<int32_t>(n);
}

template <typename T = void>
T *ptr(const at::Tensor *t) {
  return t == nullptr ? nullptr : static_cast<T *>(t->data_ptr());
}
template <typename T = void>
T *ptr(const at::Tensor &t) {
  return static_cast<T *>(t.data_ptr());
}

// A checked 4-bit K and V cache.
struct Q4 {
  const at::Tensor *kc, *kp, *vc, *vp;
  int32_t heads, group, block;
  int64_t blocks;
  explicit Q4(Args &a) {
    a.cache("k_cache", &kc, &kp);
    a.cache("v_cache", &vc, &vp);
    const int64_t groups = kp->size(3);
    require(kc->size(3) == 64 && (groups == 1 || groups == 2 || groups == 4) && kp->size(0) == kc->size(0) &&
            kp->size(1) == kc->size(1) && kp->size(2) == kc->size(2) && kp->size(4) == 2 &&
            vc->sizes() == kc->sizes() && vp->sizes() == kp->sizes());
    blocks = kc->size(0);
    heads = size32(*kc, 1);
    block = size32(*kc, 2);
    group = static_cast<int32_t>(128 / groups);
  }
};

constexpr auto kBf16 = at::kBFloat16;
constexpr auto kI32 = at::kInt;
constexpr auto kF32 = at::kFloat;

pkv_status kv_store_q4(Args &a) {
  const at::Tensor &k = a.tensor("k", kBf16, 3), &v = a.tensor("v", kBf16, 3);
  const Q4 c(a);
  const at::Tensor &slots = a.tensor("slot_mapping", kI32, 1);
  require(k.sizes() == v.sizes() && k.size(1) == c.heads && k.size(2) == 128 && slots.size(0) == k.size(0));
  return pkv_kv_store_q4(ptr(k), ptr(v), ptr(c.kc), ptr(c.kp), ptr(c.vc), ptr(c.vp), ptr<int32_t>(slots), size32(k, 0),
                         c.heads, 128, c.group, c.block, c.blocks, a.stream());
}

// Returns (status, k, v).
PyObject *kv_load_q4(Args &a) {
  const Q4 c(a);
  const at::Tensor &slots = a.tensor("slots", kI32, 1);
  const at::Tensor *given[2] = {a.maybe("k", kBf16, 3), a.maybe("v", kBf16, 3)};
  at::Tensor out[2];
  for (int i = 0; i < 2; ++i) {
    out[i] = given[i] != nullptr ? *given[i]
                                 : at::empty({slots.size(0), c.heads, 128}, slots.options().dtype(kBf16));
    require(out[i].size(0) == slots.size(0) && out[i].size(1) == c.heads && out[i].size(2) == 128);
  }
  const pkv_status st =
      pkv_kv_load_q4(ptr(c.kc), ptr(c.kp), ptr(c.vc), ptr(c.vp), ptr<int32_t>(slots), ptr(out[0]), ptr(out[1]),
                     size32(slots, 0), c.heads, 128, c.group, c.block, c.blocks, a.stream());
  return Py_BuildValue("(iNN)", static_cast<int>(st), THPVariable_Wrap(out[0]), THPVariable_Wrap(out[1]));
}

// The inputs and outputs that the decode calls share.
struct Decode {
  const at::Tensor &q, &tables, &lens;
  int32_t max_len;
  float scale;
  const at::Tensor &out;
  const at::Tensor *lse, *scores;
  const at::Tensor &workspace;
  int32_t window;
  explicit Decode(Args &a)
      : q(a.tensor("q", kBf16, 3)),
        tables(a.tensor("block_tables", kI32, 2)),
        lens(a.tensor("context_lens", kI32, 1)),
        max_len(a.i32("max_context_len")),
        scale(a.f32()),
        out(a.tensor("out", kBf16, 3)),
        lse(a.maybe("lse", kF32, 2)),
        scores(a.maybe("key_scores", kF32, 2)),
        workspace(a.tensor("workspace", at::kByte, 1)),
        window(a.i32("sliding_window")) {
    const int64_t S = q.size(0);
    require(q.size(2) == 128 && tables.size(0) == S && lens.size(0) == S && out.sizes() == q.sizes() &&
            (lse == nullptr || (lse->size(0) == S && lse->size(1) == q.size(1))));
    if (scores != nullptr && (scores->size(0) != S || scores->size(1) < max_len))
      fail(PyExc_ValueError, "key_scores must be [num_seqs, >= max_context_len]");
  }
};

pkv_status paged_decode_attn_q4(Args &a) {
  const Q4 c(a);
  const Decode d(a);
  return pkv_paged_decode_attn_q4(ptr(d.q), ptr(c.kc), ptr(c.kp), ptr(c.vc), ptr(c.vp), ptr<int32_t>(d.tables),
                                  size32(d.tables, 1), ptr<int32_t>(d.lens), d.max_len, size32(d.q, 0),
                                  size32(d.q, 1), c.heads, 128, c.group, c.block, c.blocks, d.scale, d.window,
                                  ptr(d.out), ptr<float>(d.lse), ptr<float>(d.scores),
                                  d.scores != nullptr ? d.scores->size(1) : 0, ptr(d.workspace),
                                  d.workspace.nbytes(), a.stream());
}

pkv_status paged_decode_attn_scores(Args &a) {
  const at::Tensor &k = a.tensor("k_cache", kBf16, 4), &v = a.tensor("v_cache", kBf16, 4);
  require(v.sizes() == k.sizes() && k.size(3) == 128);
  const Decode d(a);
  return pkv_paged_decode_attn_scores(ptr(d.q), ptr(k), ptr(v), ptr<int32_t>(d.tables), size32(d.tables, 1),
                                      ptr<int32_t>(d.lens), d.max_len, size32(d.q, 0), size32(d.q, 1), size32(k, 2),
                                      128, size32(k, 1), k.size(0), d.scale, d.window, ptr(d.out), ptr<float>(d.lse),
                                      ptr<float>(d.scores), d.scores != nullptr ? d.scores->size(1) : 0,
                                      ptr(d.workspace), d.workspace.nbytes(), a.stream());
}

pkv_status paged_prefill_attn_q4(Args &a) {
  const Q4 c(a);
  const at::Tensor &q = a.tensor("q", kBf16, 3);
  const at::Tensor &cu_q = a.tensor("cu_seqlens_q", kI32, 1), &cu_k = a.tensor("cu_seqlens_k", kI32, 1);
  const at::Tensor &tables = a.tensor("block_tables", kI32, 2);
  const int32_t max_q = a.i32("max_seqlen_q"), max_k = a.i32("max_seqlen_k"), total_k = a.i32("total_k");
  const float scale = a.f32();
  const at::Tensor &out = a.tensor("out", kBf16, 3);
  const at::Tensor *lse = a.maybe("lse", kF32, 2), *workspace = a.maybe("workspace", at::kByte, 1);
  const int32_t window = a.i32("sliding_window");
  const int64_t S = cu_q.size(0) - 1;
  require(q.size(2) == 128 && S >= 0 && cu_k.size(0) == S + 1 && tables.size(0) == S && out.sizes() == q.sizes() &&
          (lse == nullptr || (lse->size(0) == q.size(0) && lse->size(1) == q.size(1))));
  return pkv_paged_prefill_attn_q4(ptr(q), ptr(c.kc), ptr(c.kp), ptr(c.vc), ptr(c.vp), ptr<int32_t>(cu_q),
                                   ptr<int32_t>(cu_k), ptr<int32_t>(tables), size32(tables, 1),
                                   static_cast<int32_t>(S), size32(q, 0), total_k, max_q, max_k, size32(q, 1),
                                   c.heads, 128, c.group, c.block, c.blocks, scale, window, ptr(out),
                                   ptr<float>(lse), ptr(workspace), workspace != nullptr ? workspace->nbytes() : 0,
                                   a.stream());
}

// Returns (status, keep, new_lens).
PyObject *evict_select(Args &a) {
  const at::Tensor &scores = a.tensor("key_scores", kF32, 2), &lens = a.tensor("context_lens", kI32, 1);
  const int32_t budget = a.i32("budget"), recent = a.i32("recent");
  const at::Tensor *given[2] = {a.maybe("keep", kI32, 2), a.maybe("new_lens", kI32, 1)};
  const int64_t S = scores.size(0);
  require(lens.size(0) == S);
  at::Tensor keep = given[0] != nullptr ? *given[0] : at::empty({S, budget > 0 ? budget : 0}, lens.options());
  at::Tensor new_lens = given[1] != nullptr ? *given[1] : at::empty({S}, lens.options());
  require(keep.size(0) == S && keep.size(1) == (budget > 0 ? budget : 0) && new_lens.size(0) == S);
  // memory allocated here may hold an earlier step's selection
  const auto select = given[0] != nullptr && given[1] != nullptr ? pkv_evict_select : pkv_evict_select_new;
  const pkv_status st = select(ptr<float>(scores), scores.size(1), ptr<int32_t>(lens), size32(scores, 1),
                               size32(scores, 0), budget, recent, ptr<int32_t>(keep), ptr<int32_t>(new_lens),
                               a.stream());
  return Py_BuildValue("(iNN)", static_cast<int>(st), THPVariable_Wrap(keep), THPVariable_Wrap(new_lens));
}

// Tables, kept positions and scores of a compaction.
struct Compact {
  const at::Tensor &src, &dst, &keep, &new_lens;
  const at::Tensor *scores, *dst_scores;
  explicit Compact(Args &a)
      : src(a.tensor("src_tables", kI32, 2)),
        dst(a.tensor("dst_tables", kI32, 2)),
        keep(a.tensor("keep", kI32, 2)),
        new_lens(a.tensor("new_lens", kI32, 1)),
        scores(a.maybe("key_scores", kF32, 2)),
        dst_scores(a.maybe("dst_key_scores", kF32, 2)) {
    const int64_t S = src.size(0);
    require(dst.size(0) == S && keep.size(0) == S && new_lens.size(0) == S &&
            (scores == nullptr || scores->size(0) == S) && (dst_scores == nullptr || dst_scores->size(0) == S));
  }
  int64_t stride(const at::Tensor *t) const { return t != nullptr ? t->size(1) : 0; }
};

pkv_status evict_compact(Args &a) {
  const at::Tensor &k = a.tensor("k_cache", kBf16, 4), &v = a.tensor("v_cache", kBf16, 4);
  require(v.sizes() == k.sizes());
  const Compact c(a);
  return pkv_evict_compact(ptr(k), ptr(v), ptr<int32_t>(c.src), size32(c.src, 1), ptr<int32_t>(c.dst),
                           size32(c.dst, 1), ptr<int32_t>(c.keep), size32(c.keep, 1), ptr<int32_t>(c.new_lens),
                           size32(c.src, 0), size32(k, 2), size32(k, 3), size32(k, 1), k.size(0),
                           ptr<float>(c.scores), c.stride(c.scores), ptr<float>(c.dst_scores), c.stride(c.dst_scores),
                           a.stream());
}

pkv_status evict_compact_q4(Args &a) {
  const Q4 q(a);
  const Compact c(a);
  return pkv_evict_compact_q4(ptr(q.kc), ptr(q.kp), ptr(q.vc), ptr(q.vp), ptr<int32_t>(c.src), size32(c.src, 1),
                              ptr<int32_t>(c.dst), size32(c.dst, 1), ptr<int32_t>(c.keep), size32(c.keep, 1),
                              ptr<int32_t>(c.new_lens), size32(c.src, 0), q.heads, 128, q.group, q.block, q.blocks,
                              ptr<float>(c.scores), c.stride(c.scores), ptr<float>(c.dst_scores),
                              c.stride(c.dst_scores), a.stream());
}

PyObject *result(pkv_status st) { return PyLong_FromLong(static_cast<long>(st)); }
PyObject *result(PyObject *o) { return o; }

// A module function around `F` of `N` arguments: no C++ exception leaves it.
template <auto F, Py_ssize_t N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
  try {
    Args a("pkv", args, n, N);
    return result(F(a));
  } catch (const PythonError &) {
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

#define PKV_ENTRY(name, n) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<name, n>)), METH_FASTCALL, nullptr}

PyMethodDef kMethods[] = {
    PKV_ENTRY(kv_store_q4, 6),           PKV_ENTRY(kv_load_q4, 6),         PKV_ENTRY(paged_decode_attn_q4, 13),
    PKV_ENTRY(paged_decode_attn_scores, 13), PKV_ENTRY(paged_prefill_attn_q4, 15), PKV_ENTRY(evict_select, 7),
    PKV_ENTRY(evict_compact, 9),         PKV_ENTRY(evict_compact_q4, 9),   {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&kModule); }
