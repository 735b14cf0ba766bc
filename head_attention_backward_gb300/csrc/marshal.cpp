// Argument marshalling of the serving entry points (attn_rope, attn_kv_plan,
// attn_kv_append, attn_kv_fwd, attn_kv_weigh, attn_kv_evict) and of the 8-bit checkpoints (attn_checkpoint_save,
// attn_bwd_checkpoint) from torch tensors: checks, outputs, the
// parameter struct and the call, in one compiled step.  These calls take a few
// microseconds of device time; done in Python, reading some forty tensor
// attributes and allocating through the Python API took 16 to 35 us of host time.
// No arithmetic happens here.  The functions are called by binding.py, which
// documents them and turns statuses into errors.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/LegacyTypeDispatch.h>
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <ATen/ops/empty_strided.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstring>
#include <string>

#include "../../include/attn_bwd.h"

namespace {

// The C ABI's functions, from the library that binding.py loaded.
struct Entries {
  int (*rope)(const attn_rope_params*, cudaStream_t);
  int (*plan)(const attn_kv_plan_params*, cudaStream_t);
  int (*append)(const attn_kv_append_params*, cudaStream_t);
  int (*fwd_size)(const attn_kv_fwd_params*, size_t*);
  int (*fwd)(const attn_kv_fwd_params*, void*, size_t, cudaStream_t);
  int (*fwd_status)(const attn_kv_fwd_params*, const void*, size_t, cudaStream_t, int*);
  int (*ck_save)(const attn_checkpoint_params*, cudaStream_t);
  int (*ck_bwd_size)(const attn_bwd_params*, const attn_checkpoint*, size_t*);
  int (*ck_bwd)(const attn_bwd_params*, const attn_checkpoint*, void*, size_t, cudaStream_t);
  int (*bwd_status)(const void*, cudaStream_t, int*);
  int (*weigh)(const attn_kv_weigh_params*, cudaStream_t);
  int (*evict_size)(const attn_kv_evict_params*, size_t*);
  int (*evict)(const attn_kv_evict_params*, void*, size_t, cudaStream_t);
} entries;
constexpr int N_ENTRIES = sizeof(entries) / sizeof(void*);
bool bound = false;

struct Refused {
  std::string why;
};

std::string text(at::IntArrayRef s) {
  std::string r = "[";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + "]";
}

[[noreturn]] void refuse(const std::string& what, const char* want, const at::Tensor& t) {
  throw Refused{what + " must be " + want + "; got " + c10::toString(t.scalar_type()) + " " + text(t.sizes()) +
                " strides " + text(t.strides()) + " on " + t.device().str()};
}

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) throw Refused{std::string(what) + " must be a tensor"};
  return THPVariable_Unpack(o);
}

template <typename T>
T* pointer(const at::Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}

// attn_dtype_t of a tensor, or -1.
int dtype_code(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return ATTN_BF16;
    case at::kHalf: return ATTN_FP16;
    case at::kFloat: return ATTN_FP32;
    default: return -1;
  }
}

bool on(const at::Tensor& t, int index) { return t.is_cuda() && t.get_device() == index; }

// A contiguous vector of n whole numbers.
template <typename T>
T* vector(PyObject* o, const char* what, int64_t n, int index) {
  const at::Tensor& t = tensor(o, what);
  const at::ScalarType want = sizeof(T) == 8 ? at::kLong : at::kInt;
  if (t.scalar_type() != want || t.dim() != 1 || t.size(0) != n || (n > 1 && t.stride(0) != 1) || !on(t, index))
    refuse(what, (std::string("a contiguous ") + (sizeof(T) == 8 ? "int64" : "int32") + " vector of " + std::to_string(n) +
                  " on cuda:" + std::to_string(index)).c_str(), t);
  return pointer<T>(t);
}

// Three zero strides mean contiguous to the library, so an expanded tensor must
// not reach it: its first element stands for all of them.
void spread(const at::Tensor& t, const char* what) {
  for (int64_t i = 0; i < t.dim(); ++i)
    if (t.size(i) > 1 && t.stride(i) == 0) refuse(what, "a tensor that is not expanded", t);
}

// {0, row, head} strides of [T, H, D]; a dimension of one entry may carry any
// stride and is given the contiguous one.
void rows3(const at::Tensor& t, const char* what, int64_t out[3]) {
  const int64_t n = t.size(0), h = t.size(1), d = t.size(2);
  if (d > 1 && t.stride(2) != 1) refuse(what, "contiguous in the head dimension", t);
  spread(t, what);
  out[0] = 0;
  out[2] = h > 1 ? t.stride(1) : d;
  out[1] = n > 1 ? t.stride(0) : h * out[2];
}

// The library writes this tensor of the caller's: what autograd saved of it before
// no longer holds.
void changed(const at::Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();   // those have no version
}

cudaStream_t stream_of(int index) {
  if (!bound) throw Refused{"the library has not been loaded"};
  const int current = c10::cuda::current_device();
  if (index != current)
    throw Refused{"tensors on device " + std::to_string(index) + ", but the current device is " + std::to_string(current)};
  return c10::cuda::getCurrentCUDAStream(index).stream();
}

template <typename F>
int call(F f) {   // other Python threads may run meanwhile
  int st;
  Py_BEGIN_ALLOW_THREADS
  st = f();
  Py_END_ALLOW_THREADS
  return st;
}

// Runs one of the functions below; no C++ exception leaves.
template <typename F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, F f) {
  if (got != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, expected %zd", got, want);
    return nullptr;
  }
  try {
    at::AutoDispatchBelowADInplaceOrView no_autograd;   // outputs are plain new tensors and views of them
    return f();
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.why.c_str());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

int64_t whole(PyObject* o, const char* what) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Refused{std::string(what) + " must be a whole number"};
  }
  return v;
}
int32_t whole32(PyObject* o, const char* what) {
  const int64_t v = whole(o, what);
  if (v < INT32_MIN || v > INT32_MAX) throw Refused{std::string(what) + " does not fit 32 bits"};
  return (int32_t)v;
}

bool truth(PyObject* o, const char* what) {
  const int t = PyObject_IsTrue(o);
  if (t < 0) {
    PyErr_Clear();
    throw Refused{std::string(what) + " must be a truth value"};
  }
  return t == 1;
}

// bind(addresses of the entries, in their order)
PyObject* py_bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, N_ENTRIES, [&]() -> PyObject* {
    void* p[N_ENTRIES];
    for (int i = 0; i < N_ENTRIES; ++i) {
      p[i] = reinterpret_cast<void*>(whole(a[i], "an address"));
      if (!p[i]) throw Refused{"a null address"};
    }
    static_assert(sizeof(p) == sizeof(entries), "one pointer per entry");
    std::memcpy(&entries, p, sizeof(p));
    bound = true;
    Py_RETURN_NONE;
  });
}

// rope(q, k or None, positions, inv_freq, pair_axis or None, interleaved, inverse,
// q_out or None, k_out or None) -> (status, q_out, k_out or None)
PyObject* py_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    const at::Tensor& q = tensor(a[0], "q");
    const bool has_k = a[1] != Py_None;
    attn_rope_params p{};
    p.dtype = dtype_code(q);
    const int64_t dims = q.dim();
    if (p.dtype < 0 || !q.is_cuda() || (dims != 3 && dims != 4) || q.stride(-1) != 1)
      refuse("q", "[T, H, D] or [B, S, H, D] in bf16, fp16 or fp32 on a GPU, contiguous in D", q);
    const int index = q.get_device();
    const int64_t rows_dims = dims - 2, rows = q.size(rows_dims - 1);
    const int64_t batch = dims == 4 ? q.size(0) : 1;
    const at::Tensor& f = tensor(a[3], "inv_freq");
    if (f.scalar_type() != at::kDouble || f.is_cuda() || f.dim() != 1 || !f.is_contiguous())
      refuse("inv_freq", "a contiguous float64 vector on the host", f);
    const int64_t half = f.size(0);
    // int32 holds what the library accepts; larger sizes are refused there or here
    if (batch > INT32_MAX || rows > INT32_MAX || q.size(-2) > INT32_MAX || q.size(-1) > INT32_MAX || half > (1 << 20))
      throw Refused{"sizes past 32 bits"};
    p.batch = (int32_t)batch;
    p.seqlen = (int32_t)rows;
    p.nhead_q = (int32_t)q.size(-2);
    p.head_dim = (int32_t)q.size(-1);
    p.rot_dim = (int32_t)(2 * half);
    p.inv_freq = pointer<const double>(f);
    if (a[4] != Py_None) {
      const at::Tensor& x = tensor(a[4], "pair_axis");
      if (x.scalar_type() != at::kByte || x.is_cuda() || x.dim() != 1 || x.size(0) != half || !x.is_contiguous())
        refuse("pair_axis", "a contiguous uint8 vector on the host, as long as inv_freq", x);
      p.pair_axis = pointer<const uint8_t>(x);
    }
    p.interleaved = truth(a[5], "interleaved");
    p.inverse = truth(a[6], "inverse");
    const at::Tensor& pos = tensor(a[2], "positions");
    const int64_t axes = pos.dim() - rows_dims;   // 0 or 1 leading dimension
    bool fits = (axes == 0 || axes == 1) && pos.scalar_type() == at::kInt && on(pos, index);
    for (int64_t i = 0; fits && i < rows_dims; ++i) fits = pos.size(axes + i) == q.size(i);
    if (!fits) refuse("positions", "int32 with the rows of q, or [axes, rows of q], next to q", pos);
    p.n_axes = axes ? (int32_t)pos.size(0) : 1;
    p.stride_pos[0] = axes ? pos.stride(0) : 0;
    p.stride_pos[1] = dims == 4 ? pos.stride(axes) : 0;
    p.stride_pos[2] = pos.stride(axes + rows_dims - 1);
    p.positions = pointer<const int32_t>(pos);
    auto strides = [&](const at::Tensor& t, const char* what, int64_t out[3]) {
      spread(t, what);
      out[0] = dims == 4 ? t.stride(0) : 0;
      out[1] = t.stride(rows_dims - 1);
      out[2] = t.stride(rows_dims);
    };
    auto like = [&](const at::Tensor& t) { return t.is_contiguous() ? at::empty(t.sizes(), t.options()) : at::empty_like(t); };
    auto output = [&](PyObject* o, const at::Tensor& t, const char* what) {
      if (o == Py_None) return like(t);
      const at::Tensor& r = tensor(o, what);
      if (r.scalar_type() != t.scalar_type() || r.sizes() != t.sizes() || !on(r, index) || r.stride(-1) != 1)
        refuse(what, "of its input's type, shape and device, contiguous in the head dimension", r);
      return r;
    };
    cudaStream_t stream = stream_of(index);
    const at::Tensor qo = output(a[7], q, "out[0]");
    p.q = q.data_ptr();
    p.q_out = qo.data_ptr();
    strides(q, "q", p.stride_q);
    strides(qo, "out[0]", p.stride_q_out);
    at::Tensor ko;
    if (has_k) {
      const at::Tensor& k = tensor(a[1], "k");
      bool same = k.scalar_type() == q.scalar_type() && on(k, index) && k.dim() == dims && k.size(-1) == q.size(-1) &&
                  k.stride(-1) == 1 && k.size(-2) <= INT32_MAX;
      for (int64_t i = 0; same && i < rows_dims; ++i) same = k.size(i) == q.size(i);
      if (!same) refuse("k", "like q but for its heads", k);
      ko = output(a[8], k, "out[1]");
      p.nhead_kv = (int32_t)k.size(-2);
      p.k = k.data_ptr();
      p.k_out = ko.data_ptr();
      strides(k, "k", p.stride_k);
      strides(ko, "out[1]", p.stride_k_out);
    }
    if (a[7] != Py_None) changed(qo);
    if (has_k && a[8] != Py_None) changed(ko);
    const int st = call([&] { return entries.rope(&p, stream); });
    return Py_BuildValue("iNN", st, THPVariable_Wrap(qo), has_k ? THPVariable_Wrap(ko) : Py_NewRef(Py_None));
  });
}

// cache(k, v, k_exp, v_exp) -> (attn_kv_cache as bytes, device, pages, page size, kv heads, d_qk, d_v)
PyObject* py_cache(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 4, [&]() -> PyObject* {
    const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
    const bool bytes = k.scalar_type() == at::kFloat8_e4m3fn || k.scalar_type() == at::kByte;
    if (!bytes || k.dim() != 4 || !k.is_cuda() || k.stride(3) != 1)
      refuse("k", "[pages, page_size, kv heads, d_qk] in float8_e4m3fn or uint8 on a GPU, contiguous in d_qk", k);
    const int index = k.get_device();
    if (v.scalar_type() != k.scalar_type() || v.dim() != 4 || v.size(0) != k.size(0) || v.size(1) != k.size(1) ||
        v.size(2) != k.size(2) || !on(v, index) || v.stride(3) != 1)
      refuse("v", "like k but for d_v", v);
    spread(k, "k");
    spread(v, "v");
    attn_kv_cache c{};
    for (int i = 0; i < 2; ++i) {
      const at::Tensor& e = tensor(a[2 + i], i ? "v_exp" : "k_exp");
      if (e.scalar_type() != at::kByte || e.dim() != 2 || e.size(0) != k.size(0) || e.size(1) != k.size(2) ||
          !on(e, index) || !e.is_contiguous())
        refuse(i ? "v_exp" : "k_exp", "contiguous uint8 [pages, kv heads] next to k", e);
      (i ? c.v_exp : c.k_exp) = pointer<uint8_t>(e);
    }
    for (int i = 0; i < 4; ++i)
      if (k.size(i) > INT32_MAX || v.size(i) > INT32_MAX) throw Refused{"sizes past 32 bits"};
    c.num_pages = (int32_t)k.size(0);
    c.page_size = (int32_t)k.size(1);
    c.nhead_kv = (int32_t)k.size(2);
    c.d_qk = (int32_t)k.size(3);
    c.d_v = (int32_t)v.size(3);
    c.k = k.data_ptr();
    c.v = v.data_ptr();
    for (int i = 0; i < 3; ++i) {
      c.stride_k[i] = k.stride(i);
      c.stride_v[i] = v.stride(i);
    }
    return Py_BuildValue("y#iiiiii", reinterpret_cast<const char*>(&c), (Py_ssize_t)sizeof(c), index, c.num_pages,
                         c.page_size, c.nhead_kv, c.d_qk, c.d_v);
  });
}

// The description that a KvCache, a tuple (k, v, k_exp, v_exp, packed, ...), keeps of
// its tensors.  Their memory may have been replaced since (set_, .data, a resized
// storage): the addresses have to be those that were packed.
void read_cache(PyObject* o, attn_kv_cache* c) {
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) < 5) throw Refused{"cache must be a KvCache"};
  PyObject* packed = PyTuple_GET_ITEM(o, 4);
  if (!PyBytes_Check(packed) || PyBytes_GET_SIZE(packed) != sizeof(*c)) throw Refused{"cache must be a KvCache"};
  std::memcpy(c, PyBytes_AS_STRING(packed), sizeof(*c));
  const void* at[4] = {c->k, c->v, c->k_exp, c->v_exp};
  for (int i = 0; i < 4; ++i)
    if (tensor(PyTuple_GET_ITEM(o, i), "a tensor of the cache").data_ptr() != at[i])
      throw Refused{"a tensor of the cache has moved since its KvCache was made: make a new one"};
}

const at::Tensor& table(PyObject* o, int64_t batch, int index, int32_t* cols, int64_t* stride) {
  const at::Tensor& t = tensor(o, "block_table");
  if (t.scalar_type() != at::kInt || t.dim() != 2 || t.size(0) != batch || t.size(1) > INT32_MAX || !on(t, index) ||
      (t.size(1) > 1 && t.stride(1) != 1))
    refuse("block_table", ("int32 [" + std::to_string(batch) + ", blocks] with contiguous rows on cuda:" +
                           std::to_string(index)).c_str(), t);
  *cols = (int32_t)t.size(1);
  *stride = batch > 1 ? t.stride(0) : t.size(1);
  return t;
}

// Entries [at, at + n) of a new vector, as a tensor on its storage (as_strided's
// dispatch five times was a third of the call's host time).
at::Tensor piece(const at::Tensor& base, int64_t at, int64_t n) {
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(base.storage()), base.key_set(), base.dtype());
  t.unsafeGetTensorImpl()->set_storage_offset(at);
  t.unsafeGetTensorImpl()->set_sizes_contiguous(n);
  return t;
}

// plan(new_lens, seqlens, block_table, free_pages, free_count, page_size, max_tokens, out or None,
// position_offsets or None)
// -> (status, (cu_seqlens, seqlens, positions, slots, free_count, status word))
PyObject* py_plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    const at::Tensor &lens = tensor(a[0], "new_lens"), &free = tensor(a[3], "free_pages");
    if (!lens.is_cuda() || lens.dim() != 1) refuse("new_lens", "an int32 vector on a GPU", lens);
    if (free.dim() != 1) refuse("free_pages", "an int32 vector next to new_lens", free);
    const int index = lens.get_device();
    const int64_t batch = lens.size(0), pages = free.size(0);
    if (batch > INT32_MAX || pages > INT32_MAX) throw Refused{"sizes past 32 bits"};
    attn_kv_plan_params p{};
    p.batch = (int32_t)batch;
    p.page_size = whole32(a[5], "page_size");
    p.num_pages = (int32_t)pages;
    p.max_tokens = whole32(a[6], "max_tokens");
    p.new_lens = vector<int32_t>(a[0], "new_lens", batch, index);
    p.seqlens = vector<int32_t>(a[1], "seqlens", batch, index);
    const at::Tensor& blocks = table(a[2], batch, index, &p.max_blocks, &p.table_stride);
    p.block_table = pointer<int32_t>(blocks);
    p.free_pages = vector<int32_t>(a[3], "free_pages", pages, index);
    p.free_count = vector<int32_t>(a[4], "free_count", 1, index);
    if (p.max_tokens < 0) throw Refused{"max_tokens must not be negative"};
    if (a[8] != Py_None) p.position_offsets = vector<int32_t>(a[8], "position_offsets", batch, index);
    cudaStream_t stream = stream_of(index);
    PyObject* out = a[7];
    at::Tensor view[6];
    if (out == Py_None) {
      // two blocks for six vectors: the words, the slots
      const int64_t at[] = {0, batch + 1, 2 * batch + 3, -1, 2 * batch + 1, 2 * batch + 2};
      const int64_t len[] = {batch + 1, batch, p.max_tokens, p.max_tokens, 1, 1};
      const at::Tensor words = at::empty({2 * batch + 3 + p.max_tokens}, lens.options());
      view[3] = at::empty({p.max_tokens}, lens.options().dtype(at::kLong));
      for (int i = 0; i < 6; ++i)
        if (i != 3) view[i] = piece(words, at[i], len[i]);
      int32_t* w = pointer<int32_t>(words);
      p.cu_seqlens = w;
      p.seqlens_out = w + at[1];
      p.positions = w + at[2];
      p.slots = pointer<int64_t>(view[3]);
      p.free_count_out = w + at[4];
      p.status = w + at[5];
    } else {
      if (!PyTuple_Check(out) || PyTuple_GET_SIZE(out) != 6) throw Refused{"out must be a KvPlan"};
      PyObject** o = &PyTuple_GET_ITEM(out, 0);
      p.cu_seqlens = vector<int32_t>(o[0], "out.cu_seqlens", batch + 1, index);
      p.seqlens_out = vector<int32_t>(o[1], "out.seqlens", batch, index);
      p.positions = vector<int32_t>(o[2], "out.positions", p.max_tokens, index);
      p.slots = vector<int64_t>(o[3], "out.slots", p.max_tokens, index);
      p.free_count_out = vector<int32_t>(o[4], "out.free_count", 1, index);
      p.status = vector<int32_t>(o[5], "out.status", 1, index);
    }
    changed(blocks);
    changed(free);
    if (a[8] != Py_None) changed(THPVariable_Unpack(a[8]));
    if (out != Py_None)
      for (int i = 0; i < 6; ++i) changed(THPVariable_Unpack(PyTuple_GET_ITEM(out, i)));
    const int st = call([&] { return entries.plan(&p, stream); });
    if (out != Py_None) return Py_BuildValue("iO", st, out);
    return Py_BuildValue("i(NNNNNN)", st, THPVariable_Wrap(view[0]), THPVariable_Wrap(view[1]), THPVariable_Wrap(view[2]),
                         THPVariable_Wrap(view[3]), THPVariable_Wrap(view[4]), THPVariable_Wrap(view[5]));
  });
}

bool is16(const at::Tensor& t) { return t.scalar_type() == at::kBFloat16 || t.scalar_type() == at::kHalf; }

// append(k, v, slots, KvCache, device) -> status
PyObject* py_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 5, [&]() -> PyObject* {
    const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
    const int index = whole32(a[4], "device");
    attn_kv_append_params p{};
    read_cache(a[3], &p.cache);
    if (!is16(k) || k.dim() != 3 || k.size(0) > INT32_MAX || k.size(1) != p.cache.nhead_kv || k.size(2) != p.cache.d_qk ||
        !on(k, index))
      refuse("k", "bf16 or fp16 [T, kv heads, d_qk] next to the cache", k);
    if (v.scalar_type() != k.scalar_type() || v.dim() != 3 || v.size(0) != k.size(0) || v.size(1) != p.cache.nhead_kv ||
        v.size(2) != p.cache.d_v || !on(v, index))
      refuse("v", "[T, kv heads, d_v] like k", v);
    p.dtype = dtype_code(k);
    p.tokens = (int32_t)k.size(0);
    p.k = k.data_ptr();
    p.v = v.data_ptr();
    rows3(k, "k", p.stride_k);
    rows3(v, "v", p.stride_v);
    p.slots = vector<int64_t>(a[2], "slots", k.size(0), index);
    cudaStream_t stream = stream_of(index);
    for (int i = 0; i < 4; ++i) changed(THPVariable_Unpack(PyTuple_GET_ITEM(a[3], i)));
    return PyLong_FromLong(call([&] { return entries.append(&p, stream); }));
  });
}

// attend(q, KvCache, device, block_table, seqlens_k, cu_seqlens_q, cu_seqlens_q_padded or None, scale, mask,
// left, right, max_seqlen_q, max_seqlen_k, o or None, lse or None, workspace or None, check)
// -> (status, step that gave it, o, lse); steps: 0 size, 1 launch, 2 reading the device's status, 3 that status
PyObject* py_attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 17, [&]() -> PyObject* {
    const at::Tensor &q = tensor(a[0], "q"), &lens = tensor(a[4], "seqlens_k");
    const int index = whole32(a[2], "device");
    attn_kv_fwd_params p{};
    read_cache(a[1], &p.cache);
    if (!is16(q) || q.dim() != 3 || q.size(0) > INT32_MAX || q.size(1) > INT32_MAX || q.size(2) != p.cache.d_qk ||
        !on(q, index))
      refuse("q", "bf16 or fp16 [T, Hq, d_qk] next to the cache", q);
    if (lens.dim() != 1 || lens.size(0) >= INT32_MAX) refuse("seqlens_k", "an int32 vector", lens);
    const int64_t t = q.size(0), hq = q.size(1), batch = lens.size(0);
    p.dtype = dtype_code(q);
    p.batch = (int32_t)batch;
    p.nhead_q = (int32_t)hq;
    p.total_q = (int32_t)t;
    p.mask = whole32(a[8], "mask");
    p.window_left = whole32(a[9], "left");
    p.window_right = whole32(a[10], "right");
    p.max_seqlen_q = whole32(a[11], "max_seqlen_q");
    p.max_seqlen_k = whole32(a[12], "max_seqlen_k");
    const double scale = PyFloat_AsDouble(a[7]);
    if (scale == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      throw Refused{"scale must be a number"};
    }
    p.softmax_scale = (float)scale;
    p.block_table = pointer<const int32_t>(table(a[3], batch, index, &p.max_blocks, &p.table_stride));
    p.seqlens_k = vector<int32_t>(a[4], "seqlens_k", batch, index);
    p.cu_seqlens_q = vector<int32_t>(a[5], "cu_seqlens_q", batch + 1, index);
    if (a[6] != Py_None) p.cu_seqlens_q_padded = vector<int32_t>(a[6], "cu_seqlens_q_padded", batch + 1, index);
    p.q = q.data_ptr();
    rows3(q, "q", p.stride_q);
    cudaStream_t stream = stream_of(index);
    at::Tensor o, lse, ws;
    if (a[13] == Py_None) {
      o = at::empty({t, hq, p.cache.d_v}, q.options());
      lse = at::empty({hq, t}, q.options().dtype(at::kFloat));
    } else {
      o = tensor(a[13], "out[0]");
      lse = tensor(a[14], "out[1]");
      if (o.scalar_type() != q.scalar_type() || o.dim() != 3 || o.size(0) != t || o.size(1) != hq ||
          o.size(2) != p.cache.d_v || !on(o, index))
        refuse("out[0]", "[T, Hq, d_v] in q's type next to it", o);
      if (lse.scalar_type() != at::kFloat || lse.dim() != 2 || lse.size(0) != hq || lse.size(1) != t || !on(lse, index) ||
          !lse.is_contiguous())
        refuse("out[1]", "contiguous float32 [Hq, T] next to q", lse);
    }
    p.o = o.data_ptr();
    rows3(o, "out[0]", p.stride_o);
    p.lse = pointer<float>(lse);
    auto result = [&](int st, int step) {
      return Py_BuildValue("iiNN", st, step, THPVariable_Wrap(o), THPVariable_Wrap(lse));
    };
    const bool check = truth(a[16], "check_status");
    size_t need = 0;
    int st = entries.fwd_size(&p, &need);
    if (st != ATTN_OK) return result(st, 0);
    if (a[15] == Py_None) {
      ws = at::empty({(int64_t)need}, q.options().dtype(at::kByte));
    } else {
      ws = tensor(a[15], "workspace");
      if (ws.scalar_type() != at::kByte || !on(ws, index) || !ws.is_contiguous())
        refuse("workspace", "a contiguous uint8 tensor next to q", ws);
    }
    const size_t bytes = (size_t)ws.numel();
    if (a[13] != Py_None) {
      changed(o);
      changed(lse);
    }
    st = call([&] { return entries.fwd(&p, ws.data_ptr(), bytes, stream); });
    if (st != ATTN_OK || !check) return result(st, 1);
    int found = ATTN_OK;
    st = call([&] { return entries.fwd_status(&p, ws.data_ptr(), bytes, stream, &found); });
    return st != ATTN_OK ? result(st, 2) : result(found, 3);
  });
}

// KvWeights (weight, position, status) next to a cache.
void read_weights(PyObject* o, const attn_kv_cache& c, int index, attn_kv_weights* w) {
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 3) throw Refused{"weights must be a KvWeights"};
  for (int i = 0; i < 2; ++i) {
    const at::Tensor& t = tensor(PyTuple_GET_ITEM(o, i), i ? "weights.position" : "weights.weight");
    if (t.scalar_type() != (i ? at::kInt : at::kFloat) || t.dim() != 3 || t.size(0) != c.num_pages ||
        t.size(1) != c.nhead_kv || t.size(2) != c.page_size || !on(t, index) || !t.is_contiguous())
      refuse(i ? "weights.position" : "weights.weight",
             i ? "contiguous int32 [pages, kv heads, page_size] next to the cache"
               : "contiguous float32 [pages, kv heads, page_size] next to the cache", t);
    (i ? *reinterpret_cast<void**>(&w->position) : *reinterpret_cast<void**>(&w->weight)) = t.data_ptr();
  }
  w->status = vector<int32_t>(PyTuple_GET_ITEM(o, 2), "weights.status", 1, index);
}

float number(PyObject* o, const char* what) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Refused{std::string(what) + " must be a number"};
  }
  return (float)v;
}

// weigh(q, lse, KvCache, device, KvWeights, block_table, seqlens_k, cu_seqlens_q, cu_seqlens_q_padded or None,
// position_offsets or None, new_lens or None, scale, mask, left, right, decay, max_seqlen_q, max_seqlen_k) -> status
PyObject* py_weigh(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 18, [&]() -> PyObject* {
    const at::Tensor &q = tensor(a[0], "q"), &lse = tensor(a[1], "lse"), &lens = tensor(a[6], "seqlens_k");
    const int index = whole32(a[3], "device");
    attn_kv_weigh_params p{};
    read_cache(a[2], &p.cache);
    read_weights(a[4], p.cache, index, &p.weights);
    if (!is16(q) || q.dim() != 3 || q.size(0) > INT32_MAX || q.size(1) > INT32_MAX || q.size(2) != p.cache.d_qk ||
        !on(q, index))
      refuse("q", "bf16 or fp16 [T, Hq, d_qk] next to the cache", q);
    if (lens.dim() != 1 || lens.size(0) >= INT32_MAX) refuse("seqlens_k", "an int32 vector", lens);
    const int64_t t = q.size(0), hq = q.size(1), batch = lens.size(0);
    if (lse.scalar_type() != at::kFloat || lse.dim() != 2 || lse.size(0) != hq || lse.size(1) != t || !on(lse, index) ||
        !lse.is_contiguous())
      refuse("lse", "contiguous float32 [Hq, T] next to q", lse);
    p.dtype = dtype_code(q);
    p.batch = (int32_t)batch;
    p.nhead_q = (int32_t)hq;
    p.total_q = (int32_t)t;
    p.block_table = pointer<const int32_t>(table(a[5], batch, index, &p.max_blocks, &p.table_stride));
    p.seqlens_k = vector<int32_t>(a[6], "seqlens_k", batch, index);
    p.cu_seqlens_q = vector<int32_t>(a[7], "cu_seqlens_q", batch + 1, index);
    if (a[8] != Py_None) p.cu_seqlens_q_padded = vector<int32_t>(a[8], "cu_seqlens_q_padded", batch + 1, index);
    if (a[9] != Py_None) p.position_offsets = vector<int32_t>(a[9], "position_offsets", batch, index);
    if (a[10] != Py_None) p.new_lens = vector<int32_t>(a[10], "new_lens", batch, index);
    p.softmax_scale = number(a[11], "scale");
    p.mask = whole32(a[12], "mask");
    p.window_left = whole32(a[13], "left");
    p.window_right = whole32(a[14], "right");
    p.decay = number(a[15], "decay");
    p.max_seqlen_q = whole32(a[16], "max_seqlen_q");
    p.max_seqlen_k = whole32(a[17], "max_seqlen_k");
    p.q = q.data_ptr();
    p.lse = pointer<const float>(lse);
    rows3(q, "q", p.stride_q);
    cudaStream_t stream = stream_of(index);
    for (int i = 0; i < 3; ++i) changed(THPVariable_Unpack(PyTuple_GET_ITEM(a[4], i)));
    return PyLong_FromLong(call([&] { return entries.weigh(&p, stream); }));
  });
}

// evict(KvCache, device, KvWeights, keep, seqlens, position_offsets, block_table, free_pages, free_count, sink, recent,
// slack, max_seqlen_k, out or None, workspace or None)
// -> (status, step that gave it, (seqlens, position_offsets, free_count, status word)); steps: 0 size, 1 launch
PyObject* py_evict(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 15, [&]() -> PyObject* {
    const at::Tensor &lens = tensor(a[4], "seqlens"), &free = tensor(a[7], "free_pages");
    const int index = whole32(a[1], "device");
    attn_kv_evict_params p{};
    read_cache(a[0], &p.cache);
    read_weights(a[2], p.cache, index, &p.weights);
    if (lens.dim() != 1 || lens.size(0) > INT32_MAX) refuse("seqlens", "an int32 vector", lens);
    const int64_t batch = lens.size(0);
    p.batch = (int32_t)batch;
    p.keep = vector<int32_t>(a[3], "keep", batch, index);
    p.seqlens = vector<int32_t>(a[4], "seqlens", batch, index);
    p.position_offsets = vector<int32_t>(a[5], "position_offsets", batch, index);
    p.block_table = pointer<const int32_t>(table(a[6], batch, index, &p.max_blocks, &p.table_stride));
    p.free_pages = vector<int32_t>(a[7], "free_pages", p.cache.num_pages, index);
    p.free_count = vector<int32_t>(a[8], "free_count", 1, index);
    p.sink = whole32(a[9], "sink");
    p.recent = whole32(a[10], "recent");
    p.slack = whole32(a[11], "slack");
    p.max_seqlen_k = whole32(a[12], "max_seqlen_k");
    cudaStream_t stream = stream_of(index);
    PyObject* out = a[13];
    at::Tensor view[4];
    if (out == Py_None) {
      const int64_t at[] = {0, batch, 2 * batch, 2 * batch + 1}, len[] = {batch, batch, 1, 1};
      const at::Tensor words = at::empty({2 * batch + 2}, lens.options());
      for (int i = 0; i < 4; ++i) view[i] = piece(words, at[i], len[i]);
      int32_t* w = pointer<int32_t>(words);
      p.seqlens_out = w;
      p.position_offsets_out = w + at[1];
      p.free_count_out = w + at[2];
      p.status = w + at[3];
    } else {
      if (!PyTuple_Check(out) || PyTuple_GET_SIZE(out) != 4) throw Refused{"out must be a KvEviction"};
      PyObject** o = &PyTuple_GET_ITEM(out, 0);
      p.seqlens_out = vector<int32_t>(o[0], "out.seqlens", batch, index);
      p.position_offsets_out = vector<int32_t>(o[1], "out.position_offsets", batch, index);
      p.free_count_out = vector<int32_t>(o[2], "out.free_count", 1, index);
      p.status = vector<int32_t>(o[3], "out.status", 1, index);
    }
    auto result = [&](int st, int step) {
      if (out != Py_None) return Py_BuildValue("iiO", st, step, out);
      return Py_BuildValue("ii(NNNN)", st, step, THPVariable_Wrap(view[0]), THPVariable_Wrap(view[1]),
                           THPVariable_Wrap(view[2]), THPVariable_Wrap(view[3]));
    };
    size_t need = 0;
    const int st = entries.evict_size(&p, &need);
    if (st != ATTN_OK) return result(st, 0);
    at::Tensor ws;
    if (a[14] == Py_None) {
      ws = at::empty({(int64_t)need}, lens.options().dtype(at::kByte));
    } else {
      ws = tensor(a[14], "workspace");
      if (ws.scalar_type() != at::kByte || !on(ws, index) || !ws.is_contiguous())
        refuse("workspace", "a contiguous uint8 tensor next to the cache", ws);
    }
    for (int i = 0; i < 4; ++i) changed(THPVariable_Unpack(PyTuple_GET_ITEM(a[0], i)));
    for (int i = 0; i < 2; ++i) changed(THPVariable_Unpack(PyTuple_GET_ITEM(a[2], i)));
    changed(free);
    if (out != Py_None)
      for (int i = 0; i < 4; ++i) changed(THPVariable_Unpack(PyTuple_GET_ITEM(out, i)));
    const size_t bytes = (size_t)ws.numel();
    return result(call([&] { return entries.evict(&p, ws.data_ptr(), bytes, stream); }), 1);
  });
}

// ------------------------------------------------------------ checkpoints

// Dimensions of a [B, S, H, D] or [T, H, D] tensor in the order of its memory, the
// last one apart, outermost first.
void memory_order(const at::Tensor& t, int order[3]) {
  const int n = (int)t.dim() - 1;
  for (int i = 0; i < n; ++i) order[i] = i;
  for (int i = 1; i < n; ++i)
    for (int j = i; j > 0 && t.stride(order[j - 1]) < t.stride(order[j]); --j) std::swap(order[j - 1], order[j]);
}

// {batch, row, head} strides of a [B, S, H, D] or [T, H, D] tensor with contiguous heads.
void strides3(const at::Tensor& t, const char* what, int64_t out[3]) {
  if (t.size(-1) > 1 && t.stride(-1) != 1) refuse(what, "contiguous in the head dimension", t);
  spread(t, what);
  out[0] = t.dim() == 4 ? t.stride(0) : 0;
  out[1] = t.stride(-3);
  out[2] = t.stride(-2);
}

// {batch, rows, heads} of one, as 32-bit sizes.
void sizes3(const at::Tensor& t, int32_t* batch, int32_t* rows, int32_t* heads) {
  for (int64_t i = 0; i < t.dim(); ++i)
    if (t.size(i) > INT32_MAX) throw Refused{"sizes past 32 bits"};
  *batch = t.dim() == 4 ? (int32_t)t.size(0) : 1;
  *rows = (int32_t)t.size(-3);
  *heads = (int32_t)t.size(-2);
}

const char* const CK_NAMES[4] = {"q", "k", "v", "o"};

// q, k, v and o of one problem: the same number of dimensions and device, k's rows v's,
// q's o's.  type: of all four, or undefined for whatever q has.
void ck_shapes(const at::Tensor* const x[4], at::ScalarType type, int index) {
  const at::Tensor& q = *x[0];
  for (int i = 0; i < 4; ++i) {
    const at::Tensor& t = *x[i];
    const at::Tensor& rows = *x[i == 2 ? 1 : 0];
    bool fits = t.scalar_type() == type && t.dim() == q.dim() && on(t, index) && (q.dim() == 3 || q.dim() == 4) &&
                t.size(-1) == x[i < 2 ? 0 : 2]->size(-1) && (q.dim() == 3 || t.size(0) == q.size(0));
    if (fits && i >= 2) fits = t.size(-3) == rows.size(-3) && t.size(-2) == rows.size(-2);
    if (!fits) refuse(CK_NAMES[i], "[B, S, H, D] or [T, H, D] of one problem, one type and one device", t);
  }
}

// The tensors of an AttnCheckpoint.
void read_checkpoint(PyObject* o, const at::Tensor* n[4], const at::Tensor* exp[4], attn_checkpoint* c) {
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 8) throw Refused{"the checkpoint must be an AttnCheckpoint"};
  for (int i = 0; i < 8; ++i) (i < 4 ? n[i] : exp[i - 4]) = &tensor(PyTuple_GET_ITEM(o, i), "a tensor of the checkpoint");
  if (!n[0]->is_cuda()) refuse("q of the checkpoint", "on a GPU", *n[0]);
  const int index = n[0]->get_device();
  ck_shapes(n, at::kChar, index);
  int64_t* strides[4] = {c->stride_q, c->stride_k, c->stride_v, c->stride_o};
  int8_t** to[4] = {&c->q, &c->k, &c->v, &c->o};
  uint8_t** exps[4] = {&c->q_exp, &c->k_exp, &c->v_exp, &c->o_exp};
  for (int i = 0; i < 4; ++i) {
    const at::Tensor &x = *n[i], &e = *exp[i];
    strides3(x, CK_NAMES[i], strides[i]);
    *to[i] = pointer<int8_t>(x);
    bool fits = e.scalar_type() == at::kByte && e.dim() == x.dim() && on(e, index) &&
                e.size(-1) * ATTN_CKPT_GROUP == x.size(-1) && (e.size(-1) <= 1 || e.stride(-1) == 1);
    for (int64_t d = 0; fits && d + 1 < x.dim(); ++d)
      fits = e.size(d) == x.size(d) && (x.size(d) <= 1 || e.stride(d) * ATTN_CKPT_GROUP == x.stride(d));
    if (!fits) refuse(std::string(CK_NAMES[i]) + "_exp", "uint8, an entry per 32 numbers in their order", e);
    *exps[i] = pointer<uint8_t>(e);
  }
}

// checkpoint(q, k, v, o, AttnCheckpoint or None) -> (status, (its eight tensors))
PyObject* py_checkpoint(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  return guarded(nargs, 5, [&]() -> PyObject* {
    const at::Tensor* x[4];
    for (int i = 0; i < 4; ++i) x[i] = &tensor(a[i], CK_NAMES[i]);
    attn_checkpoint_params p{};
    p.dtype = dtype_code(*x[0]);
    if (p.dtype < 0 || !x[0]->is_cuda()) refuse("q", "bf16, fp16 or fp32 on a GPU", *x[0]);
    const int index = x[0]->get_device();
    ck_shapes(x, x[0]->scalar_type(), index);
    int32_t rows_o, heads_o;
    sizes3(*x[0], &p.batch, &p.seqlen_q, &p.nhead_q);
    sizes3(*x[1], &p.batch, &p.seqlen_k, &p.nhead_kv);
    sizes3(*x[3], &p.batch, &rows_o, &heads_o);
    for (int i = 0; i < 4; i += 2) {
      const int64_t d = x[i]->size(-1);
      if (d > 256) return Py_BuildValue("iO", (int)ATTN_ERR_UNSUPPORTED_HEADDIM, Py_None);
      (i ? p.d_v : p.d_qk) = (int32_t)d;
    }
    int64_t* from[4] = {p.stride_q, p.stride_k, p.stride_v, p.stride_o};
    const void** at_[4] = {&p.q, &p.k, &p.v, &p.o};
    for (int i = 0; i < 4; ++i) {
      strides3(*x[i], CK_NAMES[i], from[i]);
      *at_[i] = x[i]->data_ptr();
    }
    if (p.d_qk % ATTN_CKPT_GROUP || p.d_v % ATTN_CKPT_GROUP || p.d_qk < 1 || p.d_v < 1)
      return Py_BuildValue("iO", (int)ATTN_ERR_UNSUPPORTED_HEADDIM, Py_None);
    cudaStream_t stream = stream_of(index);
    if (a[4] != Py_None) {
      const at::Tensor *n[4], *exp[4];
      read_checkpoint(a[4], n, exp, &p.ckpt);
      for (int i = 0; i < 4; ++i) {
        if (n[i]->sizes() != x[i]->sizes() || !on(*n[i], index)) refuse(std::string("out.") + CK_NAMES[i], "of its input's shape, next to it", *n[i]);
        changed(*n[i]);
        changed(*exp[i]);
      }
      return Py_BuildValue("iO", call([&] { return entries.ck_save(&p, stream); }), a[4]);
    }
    // one block for the eight tensors, which live and die together
    int64_t begin[8], total = 0;
    for (int i = 0; i < 8; ++i) {
      begin[i] = total;
      total += (x[i & 3]->numel() / (i < 4 ? 1 : ATTN_CKPT_GROUP) + 255) & ~255LL;
    }
    const at::Tensor block = at::empty({total}, x[0]->options().dtype(at::kByte));
    uint8_t* bytes = pointer<uint8_t>(block);
    int8_t** numbers[4] = {&p.ckpt.q, &p.ckpt.k, &p.ckpt.v, &p.ckpt.o};
    uint8_t** exps[4] = {&p.ckpt.q_exp, &p.ckpt.k_exp, &p.ckpt.v_exp, &p.ckpt.o_exp};
    int64_t* strides[4] = {p.ckpt.stride_q, p.ckpt.stride_k, p.ckpt.stride_v, p.ckpt.stride_o};
    at::Tensor made[8];
    for (int i = 0; i < 8; ++i) {
      const at::Tensor& s = *x[i & 3];
      int order[3];
      memory_order(s, order);
      const int64_t last = s.size(-1) / (i < 4 ? 1 : ATTN_CKPT_GROUP), dims = s.dim();
      int64_t size[4], stride[4], next = last;
      size[dims - 1] = last;
      stride[dims - 1] = 1;
      for (int64_t k = dims - 2; k >= 0; --k) {
        size[order[k]] = s.size(order[k]);
        stride[order[k]] = next;
        next *= std::max<int64_t>(1, s.size(order[k]));
      }
      made[i] = at::detail::make_tensor<c10::TensorImpl>(
          c10::Storage(block.storage()), block.key_set(), caffe2::TypeMeta::fromScalarType(i < 4 ? at::kChar : at::kByte));
      made[i].unsafeGetTensorImpl()->set_storage_offset(begin[i]);
      made[i].unsafeGetTensorImpl()->set_sizes_and_strides(at::IntArrayRef(size, dims), at::IntArrayRef(stride, dims));
      if (i < 4) {
        *numbers[i] = reinterpret_cast<int8_t*>(bytes + begin[i]);
        strides[i][0] = dims == 4 ? stride[0] : 0;
        strides[i][1] = stride[dims - 3];
        strides[i][2] = stride[dims - 2];
      } else {
        *exps[i - 4] = bytes + begin[i];
      }
    }
    const int status = call([&] { return entries.ck_save(&p, stream); });
    PyObject* out = PyTuple_New(8);
    for (int i = 0; i < 8; ++i) PyTuple_SET_ITEM(out, i, THPVariable_Wrap(made[i]));
    return Py_BuildValue("iN", status, out);
  });
}

// backward(AttnCheckpoint, do, lse, scale, mask, left, right, deterministic, cu_seqlens_q or None, cu_seqlens_k,
// max_seqlen_q, max_seqlen_k, cu_seqlens_q_padded or None, cu_seqlens_k_padded or None, workspace or None,
// dq or None, dk, dv, check, bias or None, bias type, return_dbias, dropout_p, seed or None, offset or None)
// -> (status, step that gave it, dq, dk, dv, dbias or None); steps as attend's
PyObject* py_backward(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  return guarded(nargs, 25, [&]() -> PyObject* {
    const at::Tensor *n[4], *exp[4];
    attn_checkpoint c{};
    read_checkpoint(a[0], n, exp, &c);
    const int index = n[0]->get_device();
    attn_bwd_params p{};
    int32_t batch, rows_q, rows_k;
    sizes3(*n[0], &batch, &rows_q, &p.nhead_q);
    sizes3(*n[1], &batch, &rows_k, &p.nhead_kv);
    if (n[0]->size(-1) > INT32_MAX || n[2]->size(-1) > INT32_MAX) throw Refused{"sizes past 32 bits"};
    p.d_qk = (int32_t)n[0]->size(-1);
    p.d_v = (int32_t)n[2]->size(-1);
    const bool group = a[8] != Py_None;
    if ((n[0]->dim() == 3) != group) throw Refused{"cu_seqlens_q and cu_seqlens_k go with [T, H, D] tensors"};
    if (group) {
      const at::Tensor& cu = tensor(a[8], "cu_seqlens_q");
      if (cu.dim() != 1 || cu.size(0) < 1 || cu.size(0) > INT32_MAX) refuse("cu_seqlens_q", "an int32 vector", cu);
      p.batch = (int32_t)cu.size(0) - 1;
      p.seqlen_q = whole32(a[10], "max_seqlen_q");
      p.seqlen_k = whole32(a[11], "max_seqlen_k");
      p.total_q = rows_q;
      p.total_k = rows_k;
      p.cu_seqlens_q = vector<int32_t>(a[8], "cu_seqlens_q", cu.size(0), index);
      p.cu_seqlens_k = vector<int32_t>(a[9], "cu_seqlens_k", cu.size(0), index);
      if (a[12] != Py_None) p.cu_seqlens_q_padded = vector<int32_t>(a[12], "cu_seqlens_q_padded", cu.size(0), index);
      if (a[13] != Py_None) p.cu_seqlens_k_padded = vector<int32_t>(a[13], "cu_seqlens_k_padded", cu.size(0), index);
    } else {
      if (a[9] != Py_None || a[12] != Py_None || a[13] != Py_None) throw Refused{"segment offsets need cu_seqlens_q"};
      p.batch = batch;
      p.seqlen_q = rows_q;
      p.seqlen_k = rows_k;
    }
    const at::Tensor &dout = tensor(a[1], "do"), &lse = tensor(a[2], "lse");
    p.dtype = dtype_code(dout);
    if (p.dtype < 0 || dout.sizes() != n[3]->sizes() || !on(dout, index))
      refuse("do", "bf16, fp16 or fp32, shaped like the checkpoint's o and next to it", dout);
    const bool lse_fits = lse.scalar_type() == at::kFloat && on(lse, index) && lse.is_contiguous() &&
                          (group ? lse.dim() == 2 && lse.size(0) == p.nhead_q && lse.size(1) == rows_q
                                 : lse.dim() == 3 && lse.size(0) == batch && lse.size(1) == p.nhead_q && lse.size(2) == rows_q);
    if (!lse_fits) refuse("lse", "contiguous float32 [B, Hq, S] or [Hq, T], as the forward gives it", lse);
    p.softmax_scale = number(a[3], "scale");
    p.mask = whole32(a[4], "mask");
    p.window_left = whole32(a[5], "left");
    p.window_right = whole32(a[6], "right");
    p.deterministic = whole32(a[7], "deterministic");
    p.dout = dout.data_ptr();
    p.lse = pointer<const float>(lse);
    strides3(dout, "do", p.stride_dout);
    p.dropout_p = number(a[22], "dropout_p");
    if (a[23] != Py_None) p.philox_seed = reinterpret_cast<const uint64_t*>(vector<int64_t>(a[23], "philox_seed", 1, index));
    if (a[24] != Py_None) p.philox_offset = reinterpret_cast<const uint64_t*>(vector<int64_t>(a[24], "philox_offset", 1, index));
    if (a[19] != Py_None) {
      const at::Tensor& bias = tensor(a[19], "bias");
      if (bias.scalar_type() != dout.scalar_type() || bias.dim() != 4 || bias.size(2) != rows_q || bias.size(3) != rows_k ||
          !on(bias, index) || !bias.is_contiguous())
        refuse("bias", "contiguous [1 or B, 1 or Hq, Sq, Sk] in do's type next to it", bias);
      p.bias_type = whole32(a[20], "bias type");
      p.bias = bias.data_ptr();
    }
    cudaStream_t stream = stream_of(index);
    at::Tensor g[3], dbias;
    void** to[3] = {&p.dq, &p.dk, &p.dv};
    int64_t* strides[3] = {p.stride_dq, p.stride_dk, p.stride_dv};
    static const char* const names[3] = {"out[0]", "out[1]", "out[2]"};
    for (int i = 0; i < 3; ++i) {
      if (a[15] == Py_None) {
        g[i] = at::empty_strided(n[i]->sizes(), n[i]->strides(), dout.options());
      } else {
        g[i] = tensor(a[15 + i], names[i]);
        if (g[i].scalar_type() != dout.scalar_type() || g[i].sizes() != n[i]->sizes() || !on(g[i], index))
          refuse(names[i], "in do's type, shaped like the tensor whose gradient it is", g[i]);
      }
      strides3(g[i], names[i], strides[i]);
      *to[i] = g[i].data_ptr();
    }
    if (truth(a[21], "return_dbias")) {
      dbias = at::empty({p.batch, p.nhead_q, rows_q, rows_k}, dout.options());
      p.dbias = dbias.data_ptr();
    }
    auto result = [&](int st, int step) {
      return Py_BuildValue("iiNNNN", st, step, THPVariable_Wrap(g[0]), THPVariable_Wrap(g[1]), THPVariable_Wrap(g[2]),
                           dbias.defined() ? THPVariable_Wrap(dbias) : Py_NewRef(Py_None));
    };
    size_t need = 0;
    int st = entries.ck_bwd_size(&p, &c, &need);
    if (st != ATTN_OK) return result(st, 0);
    at::Tensor ws;
    if (a[14] == Py_None) {
      ws = at::empty({(int64_t)need}, dout.options().dtype(at::kByte));
    } else {
      ws = tensor(a[14], "workspace");
      if (ws.scalar_type() != at::kByte || !on(ws, index) || !ws.is_contiguous())
        refuse("workspace", "a contiguous uint8 tensor next to do", ws);
    }
    if (a[15] != Py_None)
      for (const at::Tensor& x : g) changed(x);
    const bool check = truth(a[18], "check_status");
    const size_t bytes = (size_t)ws.numel();
    st = call([&] { return entries.ck_bwd(&p, &c, ws.data_ptr(), bytes, stream); });
    if (st != ATTN_OK || !check) return result(st, 1);
    int found = ATTN_OK;
    st = call([&] { return entries.bwd_status(ws.data_ptr(), stream, &found); });
    return st != ATTN_OK ? result(st, 2) : result(found, 3);
  });
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f))
PyMethodDef methods[] = {{"bind", FAST(py_bind), METH_FASTCALL, nullptr},     {"rope", FAST(py_rope), METH_FASTCALL, nullptr},
                         {"cache", FAST(py_cache), METH_FASTCALL, nullptr},   {"plan", FAST(py_plan), METH_FASTCALL, nullptr},
                         {"append", FAST(py_append), METH_FASTCALL, nullptr}, {"attend", FAST(py_attend), METH_FASTCALL, nullptr},
                         {"weigh", FAST(py_weigh), METH_FASTCALL, nullptr},   {"evict", FAST(py_evict), METH_FASTCALL, nullptr},
                         {"checkpoint", FAST(py_checkpoint), METH_FASTCALL, nullptr},
                         {"backward", FAST(py_backward), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&module); }
