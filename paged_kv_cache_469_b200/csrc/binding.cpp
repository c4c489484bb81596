// binding.cpp -- argument marshalling of the calls that a decode step makes many
// times: tensors to the C ABI of include/pa.h.  The kernels of such a step take a
// few microseconds; checking and passing some twenty arguments from Python took
// eight, this takes one.
//
// Each function checks what the C ABI cannot see (types, shapes, devices,
// contiguity), raises TypeError or ValueError, and else returns the C call's
// status.  Nothing is kept between calls.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "pa.h"

namespace {

struct Api {
  decltype(&pa_rope_append) rope_append = nullptr;
  decltype(&pa_rope_append_fp4) rope_append_fp4 = nullptr;
  decltype(&pa_gather_fp4) gather_fp4 = nullptr;
  decltype(&pa_attention_varlen_fp4) attention_varlen_fp4 = nullptr;
} api;

struct Refusal {
  PyObject* type;
  std::string what;
};
[[noreturn]] void refuse(PyObject* type, const std::string& what) { throw Refusal{type, what}; }
void need(bool ok, PyObject* type, const char* what) {
  if (!ok) refuse(type, what);
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refusal{nullptr, ""};
  return v;
}
int small(PyObject* o, const char* name) {
  const int64_t v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX)
    refuse(PyExc_ValueError, std::string(name) + " does not fit 32 bits");
  return (int)v;
}
int extent(const at::Tensor& t, int dim) {
  const int64_t v = t.size(dim);
  if (v > INT32_MAX) refuse(PyExc_ValueError, "a size does not fit 32 bits");
  return (int)v;
}
float number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refusal{nullptr, ""};
  return (float)v;
}
pa_dtype dtype_of(const at::Tensor& t) {
  if (t.scalar_type() == at::kFloat) return PA_DTYPE_F32;
  if (t.scalar_type() == at::kBFloat16) return PA_DTYPE_BF16;
  refuse(PyExc_TypeError, "unsupported dtype: float32 or bfloat16");
}

// The device that every tensor of a call must be on.
class Place {
 public:
  Place(const at::Tensor& t, const char* name) : first_(name), dev_(t.device()) {
    if (!t.is_cuda()) refuse(PyExc_ValueError, std::string(name) + " must be a CUDA tensor");
  }
  const Place& has(const at::Tensor& t, const char* name) const {
    if (t.device() != dev_)
      refuse(PyExc_ValueError,
             std::string(name) + " must be a CUDA tensor, on the device of " + first_);
    return *this;
  }
  const Place& whole(const at::Tensor& t, const char* name) const {
    has(t, name);
    if (!t.is_contiguous()) refuse(PyExc_ValueError, std::string(name) + " must be contiguous");
    return *this;
  }
  c10::Device device() const { return dev_; }

 private:
  const char* first_;
  c10::Device dev_;
};

// The given stream (an integer handle), or with None the device's current one.
struct CUstream_st* stream_of(PyObject* o, const c10::Device& dev) {
  if (o != Py_None) {
    void* p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) throw Refusal{nullptr, ""};
    return (struct CUstream_st*)p;
  }
  return c10::cuda::getCurrentCUDAStream(dev.index()).stream();
}

// Elements from one token's row to the next of a [tokens][heads][d] tensor whose
// rows are contiguous (a slice of a fused projection, for instance).
int64_t row_stride(const at::Tensor& t, const char* name, int64_t tokens, int64_t heads,
                   int64_t d) {
  need(t.dim() == 3 && t.size(0) == tokens && t.size(1) == heads && t.size(2) == d,
       PyExc_ValueError, "the sizes of q, k, v and the cache do not fit");
  if ((t.stride(1) != d && heads > 1) || (t.stride(2) != 1 && d > 1))
    refuse(PyExc_ValueError, std::string(name) + " must have contiguous rows");
  return tokens > 1 ? t.stride(0) : heads * d;
}

// Runs a function's body; exceptions become Python's.
template <typename Body>
PyObject* guarded(Py_ssize_t have, Py_ssize_t want, Body body) {
  if (have != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, %zd needed", have, want);
    return nullptr;
  }
  try {
    return PyLong_FromLong(body());
  } catch (const Refusal& r) {
    if (r.type) PyErr_SetString(r.type, r.what.c_str());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// A call of the C ABI, every argument read: other Python threads run meanwhile (a launch
// waits while the launch queue is full).
template <typename Call>
int unlocked(Call call) {
  PyThreadState* const state = PyEval_SaveThread();
  const int status = call();
  PyEval_RestoreThread(state);
  return status;
}

constexpr int kBlockSize = 16;

struct Fp4Cache {
  int num_blocks, heads, d;
};
Fp4Cache fp4_cache(const at::Tensor& t) {
  need(t.scalar_type() == at::kByte && t.dim() == 3 && t.size(2) % 18 == 0, PyExc_TypeError,
       "kv_cache must be uint8 [num_blocks, num_kv_heads, 18 * head_dim]");
  return Fp4Cache{extent(t, 0), extent(t, 1), extent(t, 2) / 18};
}

// Both appends.  args: q, k, v, caches (one or two), [k_scale, v_scale,]
// slot_mapping, positions, cos_sin, q_out, interleaved, stream
template <bool kFp4>
int append(PyObject* const* args) {
  const at::Tensor &q = tensor(args[0], "q"), &k = tensor(args[1], "k"), &v = tensor(args[2], "v");
  const at::Tensor& cache = tensor(args[3], kFp4 ? "kv_cache" : "k_cache");
  PyObject* const* a = args + (kFp4 ? 6 : 5);
  const at::Tensor &slots = tensor(a[0], "slot_mapping"), &q_out = tensor(a[3], "q_out");
  int num_blocks, hkv, d;
  const Place on(k, "k");
  if constexpr (kFp4) {
    const Fp4Cache c = fp4_cache(cache);
    num_blocks = c.num_blocks;
    hkv = c.heads;
    d = c.d;
    on.whole(cache, "kv_cache");
  } else {
    const at::Tensor& v_cache = tensor(args[4], "v_cache");
    need(cache.dim() == 4 && cache.size(2) == kBlockSize && v_cache.sizes() == cache.sizes(),
         PyExc_ValueError, "the caches must be [num_blocks, num_kv_heads, 16, head_dim]");
    need(cache.scalar_type() == k.scalar_type() && v_cache.scalar_type() == k.scalar_type(),
         PyExc_TypeError, "the caches must have the dtype of k");
    num_blocks = extent(cache, 0);
    hkv = extent(cache, 1);
    d = extent(cache, 3);
    on.whole(cache, "k_cache").whole(v_cache, "v_cache");
  }
  need(q.scalar_type() == k.scalar_type() && v.scalar_type() == k.scalar_type() &&
           q_out.scalar_type() == k.scalar_type(),
       PyExc_TypeError, "q, k, v and q_out must have one dtype");
  const pa_dtype dt = dtype_of(k);
  need(slots.scalar_type() == at::kLong, PyExc_TypeError, "slot_mapping must be int64");
  need(k.dim() == 3 && q.dim() == 3, PyExc_ValueError, "q and k must be [tokens, heads, head_dim]");
  const int t = extent(k, 0), hq = extent(q, 1);
  const int64_t qs = row_stride(q, "q", t, hq, d), ks = row_stride(k, "k", t, hkv, d),
                vs = row_stride(v, "v", t, hkv, d);
  need(q_out.sizes() == q.sizes() && slots.dim() == 1 && slots.size(0) == t, PyExc_ValueError,
       "the sizes of q_out or slot_mapping do not fit");
  on.has(q, "q").has(v, "v").whole(q_out, "q_out").whole(slots, "slot_mapping");
  const int64_t* positions = nullptr;
  const float* angles = nullptr;
  int64_t longest = 0;
  int rotary = 0;
  if (a[2] != Py_None) {
    need(a[1] != Py_None, PyExc_TypeError, "cos_sin needs positions");
    const at::Tensor &p = tensor(a[1], "positions"), &c = tensor(a[2], "cos_sin");
    need(p.scalar_type() == at::kLong, PyExc_TypeError, "positions must be int64");
    need(c.scalar_type() == at::kFloat && c.dim() == 2, PyExc_TypeError,
         "cos_sin must be a float32 [max_position, rotary_dim] tensor");
    need(p.dim() == 1 && p.size(0) == t, PyExc_ValueError, "the size of positions does not fit");
    on.whole(p, "positions").whole(c, "cos_sin");
    positions = (const int64_t*)p.const_data_ptr();
    angles = (const float*)c.const_data_ptr();
    longest = c.size(0);
    rotary = extent(c, 1);
  }
  const int interleaved = PyObject_IsTrue(a[4]);
  if (interleaved < 0) throw Refusal{nullptr, ""};
  c10::cuda::CUDAGuard guard(on.device());
  auto* const stream = stream_of(a[5], on.device());
  void* const to = q_out.data_ptr();
  const void *const from_q = q.const_data_ptr(), *const from_k = k.const_data_ptr(),
             *const from_v = v.const_data_ptr();
  const int64_t* const at = (const int64_t*)slots.const_data_ptr();
  void* const held = cache.data_ptr();
  if constexpr (kFp4) {
    const float k_scale = number(args[4]), v_scale = number(args[5]);
    return unlocked([&] {
      return api.rope_append_fp4(to, from_q, qs, from_k, ks, from_v, vs, held, k_scale, v_scale, at,
                                 positions, angles, longest, rotary, interleaved, t, hq, hkv, d,
                                 kBlockSize, num_blocks, dt, stream);
    });
  } else {
    void* const held_v = tensor(args[4], "v_cache").data_ptr();
    return unlocked([&] {
      return api.rope_append(to, from_q, qs, from_k, ks, from_v, vs, held, held_v, at, positions,
                             angles, longest, rotary, interleaved, t, hq, hkv, d, kBlockSize,
                             num_blocks, dt, stream);
    });
  }
}

PyObject* rope_append(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded(n, 11, [&] { return append<false>(args); });
}
PyObject* rope_append_fp4(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded(n, 12, [&] { return append<true>(args); });
}

// args: kv_cache, slots, k_scale, v_scale, k_out, v_out, stream
PyObject* gather_fp4(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded(n, 7, [&] {
    const at::Tensor &cache = tensor(args[0], "kv_cache"), &slots = tensor(args[1], "slots");
    const at::Tensor &k = tensor(args[4], "k_out"), &v = tensor(args[5], "v_out");
    const Fp4Cache c = fp4_cache(cache);
    need(slots.scalar_type() == at::kLong, PyExc_TypeError, "slots must be int64");
    need(slots.dim() == 1 && k.dim() == 3 && k.size(0) == slots.size(0) && k.size(1) == c.heads &&
             k.size(2) == c.d && v.sizes() == k.sizes(),
         PyExc_ValueError, "k_out and v_out must be [n, num_kv_heads, head_dim]");
    need(k.scalar_type() == v.scalar_type(), PyExc_TypeError, "k_out and v_out must have one dtype");
    const pa_dtype dt = dtype_of(k);
    const Place on(cache, "kv_cache");
    on.whole(cache, "kv_cache").whole(slots, "slots").whole(k, "k_out").whole(v, "v_out");
    c10::cuda::CUDAGuard guard(on.device());
    void *const to_k = k.data_ptr(), *const to_v = v.data_ptr();
    const void* const from = cache.const_data_ptr();
    const int64_t* const at = (const int64_t*)slots.const_data_ptr();
    const float k_scale = number(args[2]), v_scale = number(args[3]);
    const int n_rows = extent(slots, 0);
    auto* const stream = stream_of(args[6], on.device());
    return unlocked([&] {
      return api.gather_fp4(to_k, to_v, from, k_scale, v_scale, at, n_rows, c.heads, c.d, kBlockSize,
                            c.num_blocks, dt, stream);
    });
  });
}

// args: out, q, kv_cache, k_scale, v_scale, block_tables, seq_lens,
// query_start_loc, max_query_len, max_seq_len, scale, workspace, and the
// addresses of the host copies (int32, sizes checked by the caller) or 0, stream
PyObject* attention_varlen_fp4(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded(n, 15, [&] {
    const at::Tensor &out = tensor(args[0], "out"), &q = tensor(args[1], "q");
    const at::Tensor& cache = tensor(args[2], "kv_cache");
    const at::Tensor &tables = tensor(args[5], "block_tables"), &lens = tensor(args[6], "seq_lens");
    const at::Tensor &begins = tensor(args[7], "query_start_loc"),
                     &ws = tensor(args[11], "workspace");
    const Fp4Cache c = fp4_cache(cache);
    need(tables.scalar_type() == at::kInt && lens.scalar_type() == at::kInt &&
             begins.scalar_type() == at::kInt,
         PyExc_TypeError, "block_tables, seq_lens and query_start_loc must be int32");
    need(out.scalar_type() == q.scalar_type(), PyExc_TypeError, "out must have the dtype of q");
    const pa_dtype dt = dtype_of(q);
    need(q.dim() == 3 && q.size(2) == c.d && out.sizes() == q.sizes() && lens.dim() == 1 &&
             tables.dim() == 2 && tables.size(0) == lens.size(0) && begins.dim() == 1 &&
             begins.size(0) == lens.size(0) + 1,
         PyExc_ValueError, "the sizes of q, out, kv_cache, block_tables, seq_lens and "
                           "query_start_loc do not fit");
    const Place on(q, "q");
    on.whole(q, "q").whole(out, "out").whole(cache, "kv_cache").whole(tables, "block_tables");
    on.whole(lens, "seq_lens").whole(begins, "query_start_loc").whole(ws, "workspace");
    c10::cuda::CUDAGuard guard(on.device());
    void *const to = out.data_ptr(), *const scratch = ws.data_ptr();
    const void *const from = q.const_data_ptr(), *const held = cache.const_data_ptr();
    const int32_t *const blocks = (const int32_t*)tables.const_data_ptr(),
                  *const lengths = (const int32_t*)lens.const_data_ptr(),
                  *const starts = (const int32_t*)begins.const_data_ptr();
    const float k_scale = number(args[3]), v_scale = number(args[4]), scale = number(args[10]);
    const int wide = extent(tables, 1), seqs = extent(lens, 0), tokens = extent(q, 0),
              hq = extent(q, 1), max_query_len = small(args[8], "max_query_len"),
              max_seq_len = small(args[9], "max_seq_len");
    const auto* const lengths_host = (const int32_t*)integer(args[12]);
    const auto* const starts_host = (const int32_t*)integer(args[13]);
    const size_t scratch_bytes = ws.nbytes();
    auto* const stream = stream_of(args[14], on.device());
    return unlocked([&] {
      return api.attention_varlen_fp4(to, from, held, k_scale, v_scale, blocks, wide, lengths,
                                      starts, seqs, tokens, max_query_len, max_seq_len, hq, c.heads,
                                      c.d, kBlockSize, c.num_blocks, scale, dt, scratch,
                                      scratch_bytes, lengths_host, starts_host, stream);
    });
  });
}

// path: the library (loaded already by the caller)
PyObject* load(PyObject*, PyObject* path) {
  const char* file = PyUnicode_AsUTF8(path);
  if (!file) return nullptr;
  void* lib = dlopen(file, RTLD_NOW | RTLD_LOCAL);
  if (!lib) {
    PyErr_SetString(PyExc_RuntimeError, dlerror());
    return nullptr;
  }
  api.rope_append = (decltype(api.rope_append))dlsym(lib, "pa_rope_append");
  api.rope_append_fp4 = (decltype(api.rope_append_fp4))dlsym(lib, "pa_rope_append_fp4");
  api.gather_fp4 = (decltype(api.gather_fp4))dlsym(lib, "pa_gather_fp4");
  api.attention_varlen_fp4 =
      (decltype(api.attention_varlen_fp4))dlsym(lib, "pa_attention_varlen_fp4");
  if (!api.rope_append || !api.rope_append_fp4 || !api.gather_fp4 || !api.attention_varlen_fp4) {
    PyErr_SetString(PyExc_RuntimeError, "the library lacks a symbol: build it again");
    return nullptr;
  }
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"load", load, METH_O, nullptr},
    {"rope_append", (PyCFunction)(void*)rope_append, METH_FASTCALL, nullptr},
    {"rope_append_fp4", (PyCFunction)(void*)rope_append_fp4, METH_FASTCALL, nullptr},
    {"gather_fp4", (PyCFunction)(void*)gather_fp4, METH_FASTCALL, nullptr},
    {"attention_varlen_fp4", (PyCFunction)(void*)attention_varlen_fp4, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
