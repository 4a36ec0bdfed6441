// Python entry points of a decode loop's calls, the decode and the cache calls: tensors checked,
// outputs made, the C ABI called.
//
// Their kernels take 3 to 25 us on small batches: marshalled through ctypes with the checks in
// Python a cache call took the host 32 to 38 us (Grace) and a decode 26, more than the GPU.
// This is argument marshalling only, like _native.py, which covers the rest of the C ABI.
#include <Python.h>

#include <ATen/core/TensorBody.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <initializer_list>
#include <string>

#include "../../include/mla.h"

namespace {

PyObject* g_error = nullptr;  // MlaError(function name, status)

// a Python exception is set
struct Raised {};

[[noreturn]] void raise(PyObject* type, const std::string& what) {
  PyErr_SetString(type, what.c_str());
  throw Raised{};
}

void check(const char* fn, mla_status_t st) {
  if (st == MLA_OK) return;
  PyObject* e = g_error ? PyObject_CallFunction(g_error, "si", fn, (int)st) : nullptr;
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  } else if (!PyErr_Occurred()) {
    PyErr_SetString(PyExc_RuntimeError, fn);
  }
  throw Raised{};
}

// The library's call without the interpreter, as ctypes makes it: a launch waits while the GPU's
// queue is full.
struct Released {
  PyThreadState* held = PyEval_SaveThread();
  ~Released() { PyEval_RestoreThread(held); }
};
template <typename F>
mla_status_t unlocked(F call) {
  const Released released;
  return call();
}

std::string shape_of(const at::Tensor& t) {
  std::string s = "[";
  for (int64_t d = 0; d < t.dim(); ++d) s += (d ? ", " : "") + std::to_string(t.size(d));
  return s + "]";
}

struct Args {
  PyObject* const* a;
  int at = 0;

  const at::Tensor& tensor(const char* name) {
    PyObject* o = a[at++];
    if (!THPVariable_Check(o)) raise(PyExc_TypeError, std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
  }
  const at::Tensor* optional(const char* name) {
    if (a[at] == Py_None) {
      ++at;
      return nullptr;
    }
    return &tensor(name);
  }
  int integer() {
    const long v = PyLong_AsLong(a[at++]);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    if (v != (int)v) raise(PyExc_ValueError, "integer argument out of range");
    return (int)v;
  }
  float number() {
    const double v = PyFloat_AsDouble(a[at++]);
    if (v == -1.0 && PyErr_Occurred()) throw Raised{};
    return (float)v;
  }
  // a raw stream handle, or None: the current stream
  cudaStream_t stream() {
    PyObject* o = a[at++];
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
    void* s = PyLong_AsVoidPtr(o);
    if (!s && PyErr_Occurred()) throw Raised{};
    return static_cast<cudaStream_t>(s);
  }
};

constexpr int64_t kAny = -1;

// a dense int32 tensor of these sizes
void ints(const char* name, const at::Tensor& t, std::initializer_list<int64_t> shape) {
  if (t.scalar_type() != at::kInt) raise(PyExc_TypeError, std::string(name) + " must be int32");
  bool ok = t.dim() == (int64_t)shape.size();
  int64_t d = 0;
  for (int64_t n : shape) ok = ok && (n == kAny || n == t.size(d)), ++d;
  if (!ok) raise(PyExc_ValueError, std::string(name) + " has the wrong shape " + shape_of(t));
  if (!t.is_contiguous()) raise(PyExc_ValueError, std::string(name) + " must be contiguous");
}

void pools(const at::Tensor& ckv, const at::Tensor& kpe) {
  const auto dt = ckv.scalar_type();
  if ((dt != at::kBFloat16 && dt != at::kFloat8_e4m3fn) || kpe.scalar_type() != dt)
    raise(PyExc_TypeError, "cache pools must both be bfloat16 or float8_e4m3fn");
  if (ckv.dim() != 3 || kpe.dim() != 3 || ckv.size(2) != 512 || kpe.size(2) != 64 || kpe.size(0) != ckv.size(0) ||
      kpe.size(1) != ckv.size(1) || ckv.size(0) > INT32_MAX || ckv.size(1) > INT32_MAX)
    raise(PyExc_ValueError, "cache pools must be [pages, page_size, 512] and [pages, page_size, 64], not " +
                                shape_of(ckv) + " and " + shape_of(kpe));
  if (!ckv.is_contiguous() || !kpe.is_contiguous()) raise(PyExc_ValueError, "cache pools must be contiguous");
}

// all on one GPU, the current one: the kernels launch there
void here(std::initializer_list<const at::Tensor*> tensors) {
  int dev = -1;
  for (const at::Tensor* t : tensors) {
    if (!t) continue;
    if (!t->is_cuda()) raise(PyExc_ValueError, "the calls take CUDA tensors");
    if (dev < 0) dev = c10::cuda::current_device();
    if (t->get_device() != dev)
      raise(PyExc_ValueError, "tensor on cuda:" + std::to_string(t->get_device()) + ", but the current device is cuda:" +
                                  std::to_string(dev));
  }
}

int32_t* i32(const at::Tensor& t) { return static_cast<int32_t*>(t.data_ptr()); }
int32_t* i32(const at::Tensor* t) { return t ? i32(*t) : nullptr; }
void* raw(const at::Tensor* t) { return t ? t->data_ptr() : nullptr; }

uint32_t* status_word(const at::Tensor* t) {
  if (!t) return nullptr;
  if (t->scalar_type() != at::kInt || t->numel() < 1) raise(PyExc_TypeError, "status must be an int32 tensor of one element");
  return reinterpret_cast<uint32_t*>(t->data_ptr());
}

int rows_of(const at::Tensor& t) {
  if (t.size(0) > INT32_MAX) raise(PyExc_ValueError, "too many rows");
  return (int)t.size(0);
}

mla_cache_t layout(const at::Tensor& ckv, int64_t stride, const at::Tensor* kept = nullptr) {
  if (stride > INT32_MAX) raise(PyExc_ValueError, "page table too wide");
  return {(int)ckv.size(0), (int)ckv.size(1), (int)stride, ckv.scalar_type() == at::kBFloat16 ? MLA_BF16 : MLA_E4M3,
          i32(kept)};
}

// Outputs made here belong to the stream they are written on.
struct OnStream {
  c10::cuda::OptionalCUDAStreamGuard guard;
  OnStream(cudaStream_t s, const at::Tensor& t) {
    if (s != c10::cuda::getCurrentCUDAStream().stream())
      guard.reset_stream(c10::cuda::getStreamFromExternal(s, (c10::DeviceIndex)t.get_device()));
  }
};

at::Tensor fresh(const at::Tensor& like, std::initializer_list<int64_t> shape) {
  return at::empty(at::IntArrayRef(shape.begin(), shape.size()), like.options());
}

PyObject* tuple_of(std::initializer_list<at::Tensor> ts) {
  PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
  if (!r) throw Raised{};
  Py_ssize_t k = 0;
  for (const at::Tensor& t : ts) {
    PyObject* o = THPVariable_Wrap(t);
    if (!o) {
      Py_DECREF(r);
      throw Raised{};
    }
    PyTuple_SET_ITEM(r, k++, o);
  }
  return r;
}

// a dense tensor of at least n elements of this type (or of its bits in integers of its size)
void dense(const char* name, const at::Tensor& t, at::ScalarType type, int64_t n) {
  const auto dt = t.scalar_type();
  const int64_t bytes = (int64_t)c10::elementSize(type);
  if ((int64_t)t.element_size() != bytes)
    raise(PyExc_TypeError, std::string(name) + " has elements of " + std::to_string(t.element_size()) + " bytes, expected " +
                               std::to_string(bytes));
  if (dt != type && at::isFloatingType(dt))
    raise(PyExc_TypeError, std::string(name) + " must be " + c10::toString(type) + ", not " + c10::toString(dt));
  if (!t.is_contiguous()) raise(PyExc_ValueError, std::string(name) + " must be contiguous");
  if (t.numel() < n) raise(PyExc_ValueError, std::string(name) + " is too small: " + shape_of(t));
}

// rows of this many entries, where more than one is read
void row_stride(const char* name, const at::Tensor& t, int64_t rows, int64_t n) {
  if (rows > 1 && t.dim() > 1 && t.size(-1) != n)
    raise(PyExc_ValueError, std::string(name) + " must have rows of " + std::to_string(n) + ", not " + shape_of(t));
}

// (q_latent, q_rope, ckv, kpe, page_table, seq_lens, scale, window_left, out, lse, want_lse, workspace,
//  address of the mla_config_t, global_seq_lens, local_visible_lens, stream)
PyObject* decode(Args a) {
  const at::Tensor &ql = a.tensor("q_latent"), &qr = a.tensor("q_rope"), &pc = a.tensor("ckv"), &pk = a.tensor("kpe"),
                   &table = a.tensor("page_table"), &lens = a.tensor("seq_lens");
  const float scale = a.number();
  const int window = a.integer();
  const at::Tensor *out = a.optional("out"), *lse = a.optional("lse");
  const bool want_lse = a.integer() != 0;
  const at::Tensor& ws = a.tensor("workspace");
  const void* address = PyLong_AsVoidPtr(a.a[a.at++]);
  if (!address) raise(PyExc_ValueError, "no config");
  mla_config_t cfg = *static_cast<const mla_config_t*>(address);
  const at::Tensor *global = a.optional("global_seq_lens"), *local = a.optional("local_visible_lens");
  if (ql.dim() != 4 || ql.size(1) != cfg.seq_len_q || ql.size(3) != 512)
    raise(PyExc_ValueError, "q_latent must be [B, " + std::to_string(cfg.seq_len_q) + ", H, 512], not " + shape_of(ql));
  if (pc.dim() != 3 || pc.size(2) != 512) raise(PyExc_ValueError, "ckv must be [pages, page_size, 512], not " + shape_of(pc));
  const auto es = cfg.qkv_dtype == MLA_E4M3 ? at::kFloat8_e4m3fn : at::kBFloat16;
  const auto os = cfg.out_dtype == MLA_F32 ? at::kFloat : at::kBFloat16;
  const int64_t B = ql.size(0), H = ql.size(2), rows = B * cfg.seq_len_q * H, keys = (int64_t)cfg.num_pages * pc.size(1);
  dense("q_latent", ql, es, rows * 512);
  dense("q_rope", qr, es, rows * 64);
  dense("ckv", pc, es, keys * 512);
  dense("kpe", pk, es, keys * 64);
  dense("page_table", table, at::kInt, B * cfg.page_table_stride);
  dense("seq_lens", lens, at::kInt, B);
  if (out) dense("out", *out, os, rows * 512);
  if (lse) dense("lse", *lse, at::kFloat, rows);
  if (global) dense("global_seq_lens", *global, at::kInt, B);
  if (local) dense("local_visible_lens", *local, at::kInt, B * cfg.seq_len_q);
  // large enough, but laid out in other rows or pages
  if (qr.dim() == 4 && (qr.size(0) != B || qr.size(1) != cfg.seq_len_q || qr.size(2) != H || qr.size(3) != 64))
    raise(PyExc_ValueError, "q_rope must be [B, Sq, H, 64] beside q_latent " + shape_of(ql) + ", not " + shape_of(qr));
  if (pk.dim() == 3 && (pk.size(1) != pc.size(1) || pk.size(2) != 64))
    raise(PyExc_ValueError, "kpe must be [pages, page_size, 64] beside ckv " + shape_of(pc) + ", not " + shape_of(pk));
  row_stride("page_table", table, B, cfg.page_table_stride);
  if (local) row_stride("local_visible_lens", *local, B, cfg.seq_len_q);
  here({&ql, &qr, &pc, &pk, &table, &lens, out, lse, &ws, global, local});
  cfg.global_seq_lens = i32(global);
  cfg.local_visible_lens = i32(local);
  const cudaStream_t stream = a.stream();
  const OnStream on(stream, ql);
  const at::Tensor o = out ? *out
                           : at::empty({B, cfg.seq_len_q, H, 512}, ql.options().dtype(os));
  at::Tensor l;
  if (lse) l = *lse;
  else if (want_lse) l = at::empty({B, cfg.seq_len_q, H}, ql.options().dtype(at::kFloat));
  const int b = rows_of(ql);
  check("mla_decode", unlocked([&] {
          return mla_decode(ql.data_ptr(), qr.data_ptr(), pc.data_ptr(), pk.data_ptr(), i32(table), i32(lens), scale, window,
                            o.data_ptr(), l.defined() ? static_cast<float*>(l.data_ptr()) : nullptr, ws.data_ptr(),
                            (size_t)ws.nbytes(), stream, b, (int)H, (int)pc.size(1), &cfg);
        }));
  return tuple_of({o, l});  // an undefined tensor is None
}

// (c, kpe, ckv_cache, kpe_cache, page_table, seq_lens, token_start, norm_weight, norm_eps, rope_table,
//  rope_interleaved, kv_descale, cp_world, cp_rank, cp_interleave, global_seq_lens, status, kept, stream)
PyObject* append(Args a) {
  const at::Tensor &c = a.tensor("c"), &kpe = a.tensor("kpe"), &pc = a.tensor("ckv_cache"), &pk = a.tensor("kpe_cache"),
                   &table = a.tensor("page_table"), &lens = a.tensor("seq_lens");
  const at::Tensor *start = a.optional("token_start"), *w = a.optional("norm_weight");
  mla_append_t o{};
  o.norm_eps = a.number();
  const at::Tensor* rope = a.optional("rope_table");
  o.rope_interleaved = a.integer();
  o.kv_descale = a.number();
  o.cp_world = a.integer();
  o.cp_rank = a.integer();
  o.cp_interleave = a.integer();
  const at::Tensor *global = a.optional("global_seq_lens"), *status = a.optional("status"), *kept = a.optional("kept");
  pools(pc, pk);
  ints("seq_lens", lens, {kAny});
  const int64_t B = lens.size(0);
  ints("page_table", table, {B, kAny});
  const auto dt = c.scalar_type();
  if ((dt != at::kBFloat16 && dt != at::kFloat) || kpe.scalar_type() != dt)
    raise(PyExc_TypeError, "c and kpe must both be bfloat16 or float32");
  if (c.dim() != 2 || kpe.dim() != 2 || c.size(1) != 512 || kpe.size(1) != 64 || kpe.size(0) != c.size(0))
    raise(PyExc_ValueError, "c and kpe must be [N, 512] and [N, 64], not " + shape_of(c) + " and " + shape_of(kpe));
  if (c.stride(1) != 1 || kpe.stride(1) != 1) raise(PyExc_ValueError, "c and kpe rows must be contiguous");
  if (start) ints("token_start", *start, {B + 1});
  if (global) ints("global_seq_lens", *global, {B});
  if (kept) ints("kept", *kept, {B});
  if (w && (w->scalar_type() != dt || w->dim() != 1 || w->size(0) != 512 || !w->is_contiguous()))
    raise(PyExc_ValueError, "norm_weight must be a contiguous [512] of c's type");
  if (rope && (rope->scalar_type() != at::kFloat || rope->dim() != 2 || rope->size(1) != 64 || !rope->is_contiguous() ||
               rope->size(0) > INT32_MAX))
    raise(PyExc_ValueError, "rope_table must be a contiguous fp32 [positions, 64]");
  here({&c, &kpe, &pc, &pk, &table, &lens, start, w, rope, global, status, kept});
  // a single token's row has no next one: its stride says nothing
  const int n = rows_of(c);
  const long long cs = n > 1 ? c.stride(0) : 512, ks = n > 1 ? kpe.stride(0) : 64;
  o.in_dtype = dt == at::kBFloat16 ? MLA_BF16 : MLA_F32;
  o.norm_weight = raw(w);
  o.rope_table = static_cast<const float*>(raw(rope));
  o.rope_positions = rope ? (int)rope->size(0) : 0;
  o.global_seq_lens = i32(global);
  const mla_cache_t l = layout(pc, table.size(1), kept);
  uint32_t* word = status_word(status);
  const cudaStream_t stream = a.stream();
  check("mla_cache_append", unlocked([&] {
          return mla_cache_append(c.data_ptr(), cs, kpe.data_ptr(), ks, i32(start), n, i32(table), i32(lens), (int)B,
                                  pc.data_ptr(), pk.data_ptr(), &l, &o, word, stream);
        }));
  Py_RETURN_NONE;
}

// (page_table, seq_lens, parents, ref_count, ckv_cache, kpe_cache, workspace, new_tokens, window_left,
//  sink_tokens, page_table_out, seq_lens_out, ref_count_out, status, kept, stream)
PyObject* fork(Args a) {
  const at::Tensor &table = a.tensor("page_table"), &lens = a.tensor("seq_lens"), &parents = a.tensor("parents"),
                   &ref = a.tensor("ref_count"), &pc = a.tensor("ckv_cache"), &pk = a.tensor("kpe_cache"),
                   &ws = a.tensor("workspace");
  const at::Tensor* add = a.optional("new_tokens");
  const int window = a.integer(), sinks = a.integer();
  const at::Tensor *table_out = a.optional("page_table_out"), *lens_out = a.optional("seq_lens_out"),
                   *ref_out = a.optional("ref_count_out"), *status = a.optional("status"), *kept = a.optional("kept");
  pools(pc, pk);
  ints("page_table", table, {kAny, kAny});
  const int64_t B = table.size(0), W = table.size(1);
  ints("seq_lens", lens, {B});
  ints("parents", parents, {kAny});
  const int64_t N = parents.size(0);
  ints("ref_count", ref, {pc.size(0)});
  if (add) ints("new_tokens", *add, {N});
  if (table_out) ints("page_table_out", *table_out, {N, W});
  if (lens_out) ints("seq_lens_out", *lens_out, {N});
  if (ref_out) ints("ref_count_out", *ref_out, {pc.size(0)});
  if (kept) ints("kept", *kept, {N});
  here({&table, &lens, &parents, &ref, &pc, &pk, &ws, add, table_out, lens_out, ref_out, status, kept});
  const cudaStream_t stream = a.stream();
  const OnStream on(stream, pc);
  const at::Tensor t2 = table_out ? *table_out : fresh(table, {N, W}), l2 = lens_out ? *lens_out : fresh(lens, {N}),
                   r2 = ref_out ? *ref_out : fresh(ref, {pc.size(0)});
  const mla_cache_t l = layout(pc, W, kept);
  const int b = rows_of(table), n = rows_of(parents);
  uint32_t* word = status_word(status);
  check("mla_cache_fork", unlocked([&] {
          return mla_cache_fork(i32(table), i32(lens), b, i32(parents), i32(add), n, i32(ref), pc.data_ptr(), pk.data_ptr(), &l,
                                window, sinks, i32(t2), i32(l2), i32(r2), ws.data_ptr(), (size_t)ws.nbytes(), word, stream);
        }));
  return tuple_of({t2, l2, r2});
}

// (page_table, ref_count, ckv_cache, kpe_cache, workspace, page_table_out, ref_count_out, page_map,
//  num_used, stream)
PyObject* compact(Args a) {
  const at::Tensor &table = a.tensor("page_table"), &ref = a.tensor("ref_count"), &pc = a.tensor("ckv_cache"),
                   &pk = a.tensor("kpe_cache"), &ws = a.tensor("workspace");
  const at::Tensor *table_out = a.optional("page_table_out"), *ref_out = a.optional("ref_count_out"),
                   *map = a.optional("page_map"), *used = a.optional("num_used");
  pools(pc, pk);
  ints("page_table", table, {kAny, kAny});
  const int64_t B = table.size(0), W = table.size(1), pages = pc.size(0);
  ints("ref_count", ref, {pages});
  if (table_out) ints("page_table_out", *table_out, {B, W});
  if (ref_out) ints("ref_count_out", *ref_out, {pages});
  if (map) ints("page_map", *map, {pages});
  if (used) ints("num_used", *used, {1});
  here({&table, &ref, &pc, &pk, &ws, table_out, ref_out, map, used});
  const cudaStream_t stream = a.stream();
  const OnStream on(stream, pc);
  const at::Tensor t2 = table_out ? *table_out : fresh(table, {B, W}), r2 = ref_out ? *ref_out : fresh(ref, {pages}),
                   m2 = map ? *map : fresh(ref, {pages}), u2 = used ? *used : fresh(ref, {1});
  const mla_cache_t l = layout(pc, W);
  const int b = rows_of(table);
  check("mla_cache_compact", unlocked([&] {
          return mla_cache_compact(i32(table), b, i32(ref), pc.data_ptr(), pk.data_ptr(), &l, i32(t2), i32(r2), i32(m2), i32(u2),
                                   ws.data_ptr(), (size_t)ws.nbytes(), stream);
        }));
  return tuple_of({t2, r2, m2, u2});
}

// (ckv_cache, kpe_cache, src_pages, dst_pages, ckv_src, kpe_src, status, stream)
PyObject* copy(Args a) {
  const at::Tensor &pc = a.tensor("ckv_cache"), &pk = a.tensor("kpe_cache"), &src = a.tensor("src_pages"),
                   &dst = a.tensor("dst_pages");
  const at::Tensor *sc = a.optional("ckv_src"), *sk = a.optional("kpe_src"), *status = a.optional("status");
  pools(pc, pk);
  if (!sc != !sk) raise(PyExc_ValueError, "give both ckv_src and kpe_src, or neither");
  if (sc) {
    pools(*sc, *sk);
    if (sc->scalar_type() != pc.scalar_type() || sc->size(1) != pc.size(1))
      raise(PyExc_ValueError, "both pools must have one type and page size");
  } else {
    sc = &pc;
    sk = &pk;
  }
  ints("src_pages", src, {kAny});
  ints("dst_pages", dst, {src.size(0)});
  here({&pc, &pk, sc, sk, &src, &dst, status});
  const mla_cache_t l = layout(pc, 1);
  const int pages = rows_of(*sc), n = rows_of(src);
  uint32_t* word = status_word(status);
  const cudaStream_t stream = a.stream();
  check("mla_cache_copy", unlocked([&] {
          return mla_cache_copy(sc->data_ptr(), sk->data_ptr(), pages, pc.data_ptr(), pk.data_ptr(), i32(src), i32(dst), n, &l,
                                word, stream);
        }));
  Py_RETURN_NONE;
}

// argument count checked, C++ exceptions turned into Python's
template <PyObject* (*F)(Args), int kArgs>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != kArgs) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", kArgs, n);
    return nullptr;
  }
  try {
    return F(Args{args});
  } catch (const Raised&) {
    return nullptr;
  } catch (...) {
    torch::translate_exception_to_python(std::current_exception());  // torch's own types, out of memory among them
    return nullptr;
  }
}

PyObject* set_error(PyObject*, PyObject* type) {
  Py_INCREF(type);
  Py_XDECREF(g_error);
  g_error = type;
  Py_RETURN_NONE;
}

template <PyObject* (*F)(Args), int kArgs>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<F, kArgs>)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {
    method<decode, 16>("decode"),
    method<append, 19>("cache_append"),
    method<fork, 16>("cache_fork"),
    method<compact, 10>("cache_compact"),
    method<copy, 8>("cache_copy"),
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "mla_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_mla_binding() { return PyModule_Create(&g_module); }
