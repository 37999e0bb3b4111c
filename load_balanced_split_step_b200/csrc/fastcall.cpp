// The short way from Python into libhpcdecode for the calls of a serving loop.
//
// Checking a dozen tensors, allocating the outputs and marshalling the arguments in Python takes 15 to 25 us,
// several times the kernels of a small call. This module does the same for calls in the common form: all
// tensors plain CUDA tensors of the expected types and shapes on the current device, outside a graph
// capture where it would have to make a status word. It returns None for every other call, and when the
// library refuses one for its arguments; binding.py then goes its own way, with its checks and its messages. Nothing is
// launched before a None: an error of the launches themselves is raised here, since a second try would run a call twice
// of which a part has run.
//
// The library's functions are given by address (bind), so that another build of it can be switched to.
#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAStream.h>
#include <cuda_runtime_api.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <unordered_map>
#include <vector>

#include "hpc_decode.h"

namespace {

using at::ScalarType;
using at::Tensor;

struct Api {
  decltype(&hpc_prompt_prologue) prompt_prologue;
  decltype(&hpc_prompt_attention) prompt_attention;
  decltype(&hpc_prompt_attention_paged) prompt_attention_paged;
  decltype(&hpc_verify_drafts) verify_drafts;
  decltype(&hpc_pages_resize) pages_resize;
  decltype(&hpc_pages_fork) pages_fork;
  decltype(&hpc_pages_compact) pages_compact;
  decltype(&hpc_pages_copy) pages_copy;
  decltype(&hpc_prompt_attention_partial_bytes) partial_bytes;
} api = {};

// binding._check: raises the error of a library call, given its return code and name.
PyObject* check = nullptr;

// Thrown for whatever is not the common form.
struct NotCommon {};
// Thrown when the library could not launch.
struct NotLaunched {
  int rc;
  const char* name;
};
thread_local bool accepted = false;  // the library has taken this call: there is no other way for it any more
void require(bool ok) {
  if (!ok) throw NotCommon();
}

const Tensor& tensor(PyObject* o) {
  require(THPVariable_Check(o));
  return THPVariable_Unpack(o);
}

bool given(PyObject* o) { return o != Py_None; }

int64_t integer(PyObject* o) {
  require(PyLong_Check(o));
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    throw NotCommon();
  }
  return v;
}

int32_t int32(int64_t v) {
  require(v >= INT32_MIN && v <= INT32_MAX);
  return static_cast<int32_t>(v);
}

double number(PyObject* o) {
  require(PyFloat_Check(o) || PyLong_Check(o));
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    throw NotCommon();
  }
  return v;
}

// Other Python threads run meanwhile: a launch waits while the stream's queue is full.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  Unlocked() = default;
  Unlocked(const Unlocked&) = delete;
  ~Unlocked() { PyEval_RestoreThread(state); }
};

// One call: the device of its first tensor, its stream, and its outputs.
struct Call {
  c10::DeviceIndex dev;
  void* stream;

  explicit Call(int64_t device) : dev(static_cast<c10::DeviceIndex>(device)) {
    require(c10::cuda::current_device() == device);
    stream = c10::cuda::getCurrentCUDAStream(dev).stream();
  }
  explicit Call(const Tensor& first) : Call(first.is_cuda() ? first.get_device() : -1) {}

  // A contiguous tensor of this device and type.
  void* in(const Tensor& t, ScalarType type) const {
    require(t.is_cuda() && t.get_device() == dev && t.scalar_type() == type && t.is_contiguous());
    return t.data_ptr();
  }
  void* in(const Tensor& t, ScalarType type, at::IntArrayRef shape) const {
    require(t.sizes() == shape);
    return in(t, type);
  }
  void* optional(PyObject* o, ScalarType type, int64_t numel) const {
    if (!given(o)) return nullptr;
    const Tensor& t = tensor(o);
    require(t.numel() == numel);
    return in(t, type);
  }
  // The caller's output, or a new one.
  Tensor out(PyObject* o, ScalarType type, at::IntArrayRef shape) const {
    if (given(o)) {
      const Tensor& t = tensor(o);
      in(t, type, shape);
      return t;
    }
    return at::detail::empty_cuda(shape, type, c10::Device(c10::kCUDA, dev), std::nullopt);
  }
  // The caller's status word, or a zeroed one.
  Tensor status(PyObject* o) const {
    if (given(o)) {
      const Tensor& t = tensor(o);
      in(t, at::kInt);
      return t;
    }
    return zeroed<1, 128>();
  }
  // kWords zeroed words that nothing else has had: kTimes of them are zeroed at a time on the stream that uses
  // them, since a memset of its own for each call costs as much as a small kernel. Later calls get the others, so
  // they are plain tensors whatever mode this call runs in (inference, a dispatch mode): made without the dispatcher,
  // and not views of one another.
  template <int64_t kWords, int64_t kTimes>
  Tensor zeroed() const {
    require(c10::cuda::currentStreamCaptureStatusMayInitCtx() == c10::cuda::CaptureStatus::None);
    static auto* pieces = new std::unordered_map<void*, std::vector<Tensor>>[64];  // never freed: the driver may be gone
    require(dev < 64);
    std::vector<Tensor>& left = pieces[dev][stream];
    if (left.empty()) {
      const c10::InferenceMode normal(false);
      const Tensor all = out(Py_None, at::kInt, {kWords * kTimes});
      {
        const Unlocked unlocked;
        require(cudaMemsetAsync(all.data_ptr(), 0, all.nbytes(), static_cast<cudaStream_t>(stream)) == cudaSuccess);
      }
      for (int64_t i = 0; i < kTimes; ++i) {
        auto piece = c10::make_intrusive<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(), all.dtype());
        piece->set_sizes_contiguous({kWords});
        piece->set_storage_offset(i * kWords);
        left.emplace_back(std::move(piece));
      }
    }
    Tensor t = std::move(left.back());
    left.pop_back();
    return t;
  }
};

// Calls the library. Everything but HPC_ERR_CUDA is found before the first launch.
template <typename... P, typename... A>
void launch(const char* name, int (*f)(P...), A... args) {
  int rc;
  {
    const Unlocked unlocked;
    rc = f(args...);
  }
  if (rc == HPC_ERR_CUDA) throw NotLaunched{rc, name};
  require(rc == HPC_OK);
  accepted = true;
}

PyObject* wrap(const Tensor& t) { return THPVariable_Wrap(t); }

template <typename... T>
PyObject* tuple(const T&... t) {
  PyObject* items[] = {t.defined() ? wrap(t) : Py_NewRef(Py_None)...};
  PyObject* r = PyTuple_New(sizeof...(T));
  if (!r) return nullptr;
  for (size_t i = 0; i < sizeof...(T); ++i) PyTuple_SET_ITEM(r, i, items[i]);
  return r;
}

// Runs f; None for what is not the common form or fails before the library has it (the long way then says why).
template <typename F>
PyObject* run(Py_ssize_t n, Py_ssize_t want, F f) {
  if (n != want) Py_RETURN_NONE;
  accepted = false;
  try {
    return f();
  } catch (const NotCommon&) {
  } catch (const NotLaunched& e) {
    PyObject* r = PyObject_CallFunction(check, "is", e.rc, e.name);
    if (r) PyErr_SetString(PyExc_RuntimeError, e.name);
    Py_XDECREF(r);
    return nullptr;
  } catch (const std::exception& e) {
    if (accepted) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
      return nullptr;
    }
  }
  PyErr_Clear();
  Py_RETURN_NONE;
}

int32_t* i32(const Tensor& t) { return static_cast<int32_t*>(t.data_ptr()); }
uint32_t* word(const Tensor& t) { return reinterpret_cast<uint32_t*>(t.data_ptr()); }

// device index: a zeroed status word for a call on that device's current stream.
PyObject* status_word(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return run(n, 1, [&] {
    const Call c(integer(a[0]));
    return wrap(c.status(Py_None));
  });
}

// ---- pages
struct Pool {
  int64_t rows, max_pages, num_pages;
  const int32_t *table, *ref;
  Pool(const Call& c, const Tensor& t, const Tensor& r) {
    require(t.dim() == 2 && r.dim() == 1);
    table = static_cast<const int32_t*>(c.in(t, at::kInt));
    ref = static_cast<const int32_t*>(c.in(r, at::kInt));
    rows = t.size(0);
    max_pages = t.size(1);
    num_pages = r.size(0);
  }
};

Tensor moves_out(const Call& c, PyObject* o, int64_t capacity) {
  if (given(o)) {
    const Tensor& t = tensor(o);
    require(t.dim() == 2 && t.size(1) == 2);
    c.in(t, at::kInt);
    return t;
  }
  return c.out(o, at::kInt, {capacity > 0 ? capacity : 1, 2});
}

// table, old_lens, new_lens, ref, page_size, table_out, ref_out, moves, n_moves, status
PyObject* resize_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return run(n, 10, [&] {
    const Tensor &table = tensor(a[0]), &ref = tensor(a[3]);
    const Call c(table);
    const Pool p(c, table, ref);
    require(tensor(a[1]).numel() == p.rows && tensor(a[2]).numel() == p.rows);
    const Tensor table_out = c.out(a[5], at::kInt, {p.rows, p.max_pages}), ref_out = c.out(a[6], at::kInt, {p.num_pages}),
                 moves = moves_out(c, a[7], p.rows), count = c.out(a[8], at::kInt, {1}), status = c.status(a[9]);
    launch("hpc_pages_resize", api.pages_resize, p.table, i32(table_out), int32(p.rows), int32(p.max_pages),
           int32(integer(a[4])), static_cast<const int32_t*>(c.in(tensor(a[1]), at::kInt)),
           static_cast<const int32_t*>(c.in(tensor(a[2]), at::kInt)), p.ref, i32(ref_out), int32(p.num_pages),
           i32(moves), int32(moves.size(0)), i32(count), word(status), c.stream);
    return tuple(table_out, ref_out, moves, count, status);
  });
}

// table, lens, ref, parents, page_size, table_out, lens_out, ref_out, moves, n_moves, status
PyObject* fork_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return run(n, 11, [&] {
    const Tensor &table = tensor(a[0]), &ref = tensor(a[2]), &parents = tensor(a[3]);
    const Call c(table);
    const Pool p(c, table, ref);
    require(tensor(a[1]).numel() == p.rows);
    const int64_t rows = parents.numel();
    const Tensor table_out = c.out(a[5], at::kInt, {rows, p.max_pages}), lens_out = c.out(a[6], at::kInt, {rows}),
                 ref_out = c.out(a[7], at::kInt, {p.num_pages}), moves = moves_out(c, a[8], rows),
                 count = c.out(a[9], at::kInt, {1}), status = c.status(a[10]);
    launch("hpc_pages_fork", api.pages_fork, p.table, static_cast<const int32_t*>(c.in(tensor(a[1]), at::kInt)),
           int32(p.rows), static_cast<const int32_t*>(c.in(parents, at::kInt)), i32(table_out), i32(lens_out),
           int32(rows), int32(p.max_pages), int32(integer(a[4])), p.ref, i32(ref_out), int32(p.num_pages), i32(moves),
           int32(moves.size(0)), i32(count), word(status), c.stream);
    return tuple(table_out, ref_out, moves, count, status, lens_out);
  });
}

// table, ref, table_out, ref_out, page_map, moves, n_moves, status
PyObject* compact_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return run(n, 8, [&] {
    const Tensor &table = tensor(a[0]), &ref = tensor(a[1]);
    const Call c(table);
    const Pool p(c, table, ref);
    const Tensor table_out = c.out(a[2], at::kInt, {p.rows, p.max_pages}), ref_out = c.out(a[3], at::kInt, {p.num_pages}),
                 map = c.out(a[4], at::kInt, {p.num_pages}), moves = moves_out(c, a[5], p.num_pages / 2),
                 count = c.out(a[6], at::kInt, {1}), status = c.status(a[7]), none;
    launch("hpc_pages_compact", api.pages_compact, p.table, i32(table_out), int32(p.rows), int32(p.max_pages), p.ref,
           i32(ref_out), int32(p.num_pages), i32(map), i32(moves), int32(moves.size(0)), i32(count), word(status),
           c.stream);
    return tuple(table_out, ref_out, moves, count, status, none, map);
  });
}

// caches (a list), moves, n_moves, status
PyObject* copy_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return run(n, 4, [&] {
    const Tensor &moves = tensor(a[1]), &count = tensor(a[2]);
    const Call c(moves);
    require(PyList_Check(a[0]) && moves.dim() == 2 && moves.size(1) == 2 && count.numel() == 1);
    const Py_ssize_t caches = PyList_GET_SIZE(a[0]);
    require(caches > 0 && caches < INT32_MAX);
    const Tensor& first = tensor(PyList_GET_ITEM(a[0], 0));
    require(first.dim() >= 2 && first.size(0) > 0);
    std::vector<void*> base(caches);
    for (Py_ssize_t i = 0; i < caches; ++i) {
      const Tensor& t = tensor(PyList_GET_ITEM(a[0], i));
      require(t.element_size() == first.element_size());
      base[i] = c.in(t, t.scalar_type(), first.sizes());
    }
    const Tensor status = c.status(a[3]);
    launch("hpc_pages_copy", api.pages_copy, base.data(), static_cast<int32_t>(caches),
           first.numel() / first.size(0) * static_cast<int64_t>(first.element_size()), int32(first.size(0)),
           static_cast<const int32_t*>(c.in(moves, at::kInt)), int32(moves.size(0)),
           static_cast<const int32_t*>(c.in(count, at::kInt)), word(status), c.stream);
    return wrap(status);
  });
}

// ---- verification: draft_tokens, target_probs, draft_probs, uniforms, draft_lens, seq_lens, out_tokens, accepted,
// new_lens, status. Contiguous probabilities; padded rows go the long way.
PyObject* verify_drafts(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return run(n, 10, [&] {
    const Tensor &drafts = tensor(a[0]), &p = tensor(a[1]), &u = tensor(a[3]);
    const Call c(drafts);
    require(drafts.dim() == 2 && p.dim() == 3);
    const int64_t B = drafts.size(0), T = drafts.size(1), V = p.size(2);
    const ScalarType type = p.scalar_type();
    require(type == at::kFloat || type == at::kBFloat16);
    const void* q = given(a[2]) ? c.in(tensor(a[2]), type, {B, T, V}) : nullptr;
    const int32_t* lens = static_cast<const int32_t*>(c.optional(a[5], at::kInt, B));
    require(lens || !given(a[8]));
    const Tensor tokens = c.out(a[6], at::kInt, {B, T + 1}), accepted = c.out(a[7], at::kInt, {B}),
                 new_lens = lens ? c.out(a[8], at::kInt, {B}) : Tensor(), status = c.status(a[9]);
    launch("hpc_verify_drafts", api.verify_drafts, static_cast<const int32_t*>(c.in(drafts, at::kInt)),
           c.in(p, type, {B, T + 1, V}), V, q, V, type == at::kFloat ? HPC_FP32 : HPC_BF16,
           static_cast<const float*>(c.in(u, at::kFloat, {B, T + 1})),
           static_cast<const int32_t*>(c.optional(a[4], at::kInt, B)), lens, int32(B), int32(T), int32(V), i32(tokens),
           i32(accepted), lens ? i32(new_lens) : nullptr, word(status), c.stream);
    return tuple(tokens, accepted, new_lens, status);
  });
}

// ---- prompts
struct Cache {
  int32_t num_pages, kv_heads, page_size;
  void *k, *v;
  Cache(const Call& c, const Tensor& kp, const Tensor& vp, bool nhd, bool e4m3, int64_t head_dim) {
    require(kp.dim() == 4 && kp.size(3) == head_dim && vp.sizes() == kp.sizes());
    for (const Tensor* t : {&kp, &vp}) {
      const ScalarType type = t->scalar_type();
      require(e4m3 ? type == at::kByte || type == at::kFloat8_e4m3fn : type == at::kBFloat16);
      c.in(*t, type);
    }
    num_pages = int32(kp.size(0));
    kv_heads = int32(kp.size(nhd ? 2 : 1));
    page_size = int32(kp.size(nhd ? 1 : 2));
    k = kp.data_ptr();
    v = vp.data_ptr();
  }
};

struct Requests {
  int32_t batch, max_pages;
  const int32_t *cu, *table, *lens;
  Requests(const Call& c, const Tensor& cu_seqlens, const Tensor& block_table, const Tensor& seq_lens) {
    require(cu_seqlens.dim() == 1 && cu_seqlens.numel() >= 2 && block_table.dim() == 2);
    batch = int32(cu_seqlens.numel() - 1);
    require(block_table.size(0) == batch && seq_lens.numel() == batch);
    max_pages = int32(block_table.size(1));
    cu = static_cast<const int32_t*>(c.in(cu_seqlens, at::kInt));
    table = static_cast<const int32_t*>(c.in(block_table, at::kInt));
    lens = static_cast<const int32_t*>(c.in(seq_lens, at::kInt));
  }
};

// qkv, cu_seqlens, q_norm_w, k_norm_w, k_pages, v_pages, table, seq_lens, num_heads, kv_heads, e4m3, nhd, k_scale,
// v_scale, eps, theta, q_out, k_out, status
PyObject* prompt_prologue(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return run(n, 19, [&] {
    const Tensor& qkv = tensor(a[0]);
    const Call c(qkv);
    const int64_t Hq = integer(a[8]), Hkv = integer(a[9]);
    require(qkv.dim() == 3 && Hq > 0 && Hkv > 0 && qkv.size(1) == Hq + 2 * Hkv);
    const int64_t tokens = qkv.size(0), D = qkv.size(2);
    const bool e4m3 = integer(a[10]) != 0, nhd = integer(a[11]) != 0;
    const Cache cache(c, tensor(a[4]), tensor(a[5]), nhd, e4m3, D);
    require(cache.kv_heads == Hkv);
    const Requests r(c, tensor(a[1]), tensor(a[6]), tensor(a[7]));
    require(tensor(a[2]).numel() == D && tensor(a[3]).numel() == D);
    const float* scales[2] = {nullptr, nullptr};
    if (e4m3)
      for (int i = 0; i < 2; ++i) {
        require(given(a[12 + i]));
        scales[i] = static_cast<const float*>(c.optional(a[12 + i], at::kFloat, Hkv));
      }
    const Tensor q = c.out(a[16], at::kBFloat16, {tokens, Hq, D}), k = c.out(a[17], at::kBFloat16, {tokens, Hkv, D}),
                 status = c.status(a[18]);
    launch("hpc_prompt_prologue", api.prompt_prologue, c.in(qkv, at::kBFloat16), tokens, r.cu, r.batch,
           static_cast<const float*>(c.in(tensor(a[2]), at::kFloat)),
           static_cast<const float*>(c.in(tensor(a[3]), at::kFloat)), static_cast<float>(number(a[14])),
           static_cast<float>(number(a[15])), q.data_ptr(), k.data_ptr(), cache.k, cache.v, e4m3 ? HPC_E4M3 : HPC_BF16,
           nhd ? HPC_NHD : HPC_HND, scales[0], scales[1], cache.num_pages, cache.page_size, r.table, r.max_pages,
           r.lens, int32(Hq), int32(Hkv), int32(D), word(status), c.stream);
    return tuple(q, k, status);
  });
}

// A bf16 [tokens, heads, head_dim] view with contiguous heads.
struct Rows {
  void* at;
  int64_t tokens, heads, D, token_stride, head_stride;
  Rows(const Call& c, const Tensor& t) {
    require(t.is_cuda() && t.get_device() == c.dev && t.scalar_type() == at::kBFloat16 && t.dim() == 3 && t.stride(2) == 1);
    tokens = t.size(0);
    heads = t.size(1);
    D = t.size(2);
    token_stride = tokens > 1 ? t.stride(0) : heads * D;
    head_stride = heads > 1 ? t.stride(1) : D;
    at = t.data_ptr();
  }
};

float scale_of(PyObject* o, int64_t D) {
  return static_cast<float>(given(o) ? number(o) : 1.0 / std::sqrt(static_cast<double>(D)));
}

// Zeroed work words and, where sequences can be cut, the scratch for their parts. Both go back to the allocator
// when the call returns; it hands them out again behind this call on the stream.
struct Scratch {
  Tensor work, partial;
  Scratch(const Call& c, int64_t max_keys, int64_t head_dim) : work(c.zeroed<HPC_PROMPT_WORK_WORDS, 128>()) {
    if (max_keys > HPC_PROMPT_SPLIT_KEYS && (head_dim == 64 || head_dim == 128))
      partial = c.out(Py_None, at::kByte, {static_cast<int64_t>(api.partial_bytes(static_cast<int32_t>(head_dim)))});
  }
  void* at() const { return partial.defined() ? partial.data_ptr() : nullptr; }
  size_t bytes() const { return partial.defined() ? partial.numel() : 0; }
};

Tensor lse_out(const Call& c, PyObject* o, PyObject* wanted, const Rows& q) {
  if (!given(o) && wanted != Py_True) return Tensor();
  return c.out(o, at::kFloat, {q.tokens, q.heads});
}

// q, k, v, cu_seqlens, cu_seqlens_k, causal, sm_scale, out, lse, return_lse, status
PyObject* prompt_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return run(n, 11, [&] {
    const Call c(tensor(a[0]));
    const Rows q(c, tensor(a[0])), k(c, tensor(a[1])), v(c, tensor(a[2]));
    require(tensor(a[2]).sizes() == tensor(a[1]).sizes() && k.D == q.D);
    const Tensor& cu = tensor(a[3]);
    require(cu.dim() == 1 && cu.numel() >= 2);
    require(PyBool_Check(a[5]) && PyBool_Check(a[9]));
    if (given(a[4])) require(tensor(a[4]).dim() == 1);
    const int32_t* cu_k = static_cast<const int32_t*>(c.optional(a[4], at::kInt, cu.numel()));
    const Tensor out = c.out(a[7], at::kBFloat16, {q.tokens, q.heads, q.D}), lse = lse_out(c, a[8], a[9], q),
                 status = c.status(a[10]);
    const Scratch scratch(c, k.tokens, q.D);
    launch("hpc_prompt_attention", api.prompt_attention, q.at, q.token_stride, q.head_stride, k.at, k.token_stride,
           k.head_stride, v.at, v.token_stride, v.head_stride, q.tokens, k.tokens,
           static_cast<const int32_t*>(c.in(cu, at::kInt)), cu_k, int32(cu.numel() - 1), int32(q.heads),
           int32(k.heads), int32(q.D), a[5] == Py_True, scale_of(a[6], q.D), out.data_ptr(),
           lse.defined() ? static_cast<float*>(lse.data_ptr()) : nullptr, word(scratch.work), scratch.at(),
           scratch.bytes(), word(status), c.stream);
    return tuple(out, lse, status);
  });
}

// q, k_pages, v_pages, table, seq_lens, cu_seqlens, nhd, sm_scale, out, lse, return_lse, status
PyObject* prompt_attention_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return run(n, 12, [&] {
    const Call c(tensor(a[0]));
    const Rows q(c, tensor(a[0]));
    const bool nhd = integer(a[6]) != 0;
    const Cache cache(c, tensor(a[1]), tensor(a[2]), nhd, false, q.D);
    const Requests r(c, tensor(a[5]), tensor(a[3]), tensor(a[4]));
    require(PyBool_Check(a[10]));
    const Tensor out = c.out(a[8], at::kBFloat16, {q.tokens, q.heads, q.D}), lse = lse_out(c, a[9], a[10], q),
                 status = c.status(a[11]);
    const Scratch scratch(c, static_cast<int64_t>(r.max_pages) * cache.page_size, q.D);
    launch("hpc_prompt_attention_paged", api.prompt_attention_paged, q.at, q.token_stride, q.head_stride, cache.k,
           cache.v, HPC_BF16, nhd ? HPC_NHD : HPC_HND, cache.num_pages, cache.page_size, r.table, r.max_pages, r.lens,
           q.tokens, r.cu, r.batch, int32(q.heads), cache.kv_heads, int32(q.D), scale_of(a[7], q.D), out.data_ptr(),
           lse.defined() ? static_cast<float*>(lse.data_ptr()) : nullptr, word(scratch.work), scratch.at(),
           scratch.bytes(), word(status), c.stream);
    return tuple(out, lse, status);
  });
}

// bind(check, addresses): what raises a library call's error, and the library's functions in the order of Api.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void* f[9];
  if (n != 10) {
    PyErr_SetString(PyExc_ValueError, "bind takes a function and nine addresses");
    return nullptr;
  }
  for (int i = 0; i < 9; ++i) {
    f[i] = PyLong_AsVoidPtr(a[i + 1]);
    if (!f[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null address");
      return nullptr;
    }
  }
  Py_INCREF(a[0]);
  Py_XSETREF(check, a[0]);
  api = {reinterpret_cast<decltype(api.prompt_prologue)>(f[0]), reinterpret_cast<decltype(api.prompt_attention)>(f[1]),
         reinterpret_cast<decltype(api.prompt_attention_paged)>(f[2]), reinterpret_cast<decltype(api.verify_drafts)>(f[3]),
         reinterpret_cast<decltype(api.pages_resize)>(f[4]), reinterpret_cast<decltype(api.pages_fork)>(f[5]),
         reinterpret_cast<decltype(api.pages_compact)>(f[6]), reinterpret_cast<decltype(api.pages_copy)>(f[7]),
         reinterpret_cast<decltype(api.partial_bytes)>(f[8])};
  Py_RETURN_NONE;
}

#define ENTRY(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY(bind),          ENTRY(resize_pages),    ENTRY(fork_pages),
                         ENTRY(compact_pages), ENTRY(copy_pages),      ENTRY(verify_drafts),
                         ENTRY(prompt_prologue), ENTRY(prompt_attention), ENTRY(prompt_attention_paged),
                         ENTRY(status_word),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__fastcall() { return PyModule_Create(&module); }
