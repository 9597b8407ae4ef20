// Host side of the serving operators' Python calls: the argument checks of
// __init__.py, the output allocations and the call of the C entry point, in
// one native call.  A decode step's kernels take 1 to 3 us each (attention 20);
// these calls take the host 3 to 6 us (attention 11), the same checks from Python
// with ctypes 8 to 27.
//
// Every function returns None where an argument is not what the common case
// takes (a tensor of another type, shape, device or layout, a subclass): the
// caller then runs its own checks, which accept or name the fault.  An int is
// the C entry point's error code.  Addresses of the entry points come from
// the loaded library through bind().
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>

#include "../include/dsa_index.h"

namespace {

decltype(&dsa_block_tables) f_tables;
decltype(&dsa_index_prepare) f_prepare;
decltype(&dsa_index_prepare_fp8) f_prepare8;
decltype(&dsa_kv4_write) f_write;
decltype(&dsa_kv4_read) f_read;
decltype(&dsa_attend_kv4) f_attend;
decltype(&dsa_attend_kv4_workspace_bytes) f_attend_ws;

// The common case's tensors: on the current device and contiguous.  ok stays
// true while every argument passes.
struct Args {
  bool ok = true;
  int dev = -1;

  const at::Tensor* tensor(PyObject* o, at::ScalarType type, int64_t dim) {
    if (!ok || !THPVariable_CheckExact(o)) return fail();
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.scalar_type() != type || t.dim() != dim || !t.is_cuda() || !t.is_contiguous()) return fail();
    const int d = t.get_device();
    if (dev < 0) {
      if (d != c10::cuda::current_device()) return fail();
      dev = d;
    }
    return d == dev ? &t : fail();
  }
  // of exactly these sizes
  template <typename... S>
  void* ptr(PyObject* o, at::ScalarType type, S... sizes) {
    const at::Tensor* t = tensor(o, type, sizeof...(S));
    if (!t) return nullptr;
    const int64_t want[] = {static_cast<int64_t>(sizes)...};
    for (size_t i = 0; i < sizeof...(S); ++i)
      if (t->size(i) != want[i]) return fail(), nullptr;
    return t->data_ptr();
  }
  template <typename... S>
  void* opt(PyObject* o, at::ScalarType type, S... sizes) {
    return o == Py_None ? nullptr : ptr(o, type, sizes...);
  }
  int64_t integer(PyObject* o) {
    if (!ok || !PyLong_CheckExact(o)) return fail(), 0;
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
      PyErr_Clear();
      return fail(), 0;
    }
    return v;
  }
  void* stream() const { return c10::cuda::getCurrentCUDAStream(dev).stream(); }
  at::TensorOptions options(at::ScalarType type) const { return at::TensorOptions().dtype(type).device(at::kCUDA, dev); }

 private:
  const at::Tensor* fail() {
    ok = false;
    return nullptr;
  }
};

constexpr auto kI32 = at::kInt;
constexpr auto kBf16 = at::kBFloat16;
constexpr auto kF32 = at::kFloat;
constexpr auto kU8 = at::kByte;
constexpr int64_t kLatent = 512, kRope = 64;

bool fits_int(int64_t v) { return v >= INT32_MIN && v <= INT32_MAX; }

template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (...) {  // out of memory and the like, as torch's own calls raise them
    torch::translate_exception_to_python(std::current_exception());
    return nullptr;
  }
}

PyObject* code(int rc) { return PyLong_FromLong(rc); }

// A C entry point with the interpreter lock released: a launch can wait for room
// in the stream's queue.
template <typename F, typename... A>
int unlocked(F f, A... args) {
  PyThreadState* state = PyEval_SaveThread();
  const int rc = f(args...);
  PyEval_RestoreThread(state);
  return rc;
}

// kv4_write(latent, rope, kv_pages, slot_map, status) -> 0 or code
PyObject* kv4_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args g;
    if (n != 5) Py_RETURN_NONE;
    const at::Tensor* kv = g.tensor(a[2], kU8, 3);
    const at::Tensor* slot = g.tensor(a[3], kI32, 1);
    if (!g.ok || kv->size(2) != DSA_KV4_ENTRY_BYTES) Py_RETURN_NONE;
    const int64_t T = slot->size(0);
    void* lat = g.ptr(a[0], kBf16, T, kLatent);
    void* rope = g.ptr(a[1], kBf16, T, kRope);
    void* st = g.opt(a[4], kI32, 1);
    if (!g.ok) Py_RETURN_NONE;
    return code(unlocked(f_write, static_cast<uint16_t*>(lat), static_cast<uint16_t*>(rope), static_cast<uint8_t*>(kv->data_ptr()),
                        kv->size(0) * kv->size(1), static_cast<int32_t*>(slot->data_ptr()), T, static_cast<uint32_t*>(st),
                        g.stream()));
  });
}

// kv4_read(kv_pages, slot_map, latent_out, rope_out, status) -> 0 or code
PyObject* kv4_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args g;
    if (n != 5) Py_RETURN_NONE;
    const at::Tensor* kv = g.tensor(a[0], kU8, 3);
    const at::Tensor* slot = g.tensor(a[1], kI32, 1);
    if (!g.ok || kv->size(2) != DSA_KV4_ENTRY_BYTES) Py_RETURN_NONE;
    const int64_t T = slot->size(0);
    void* lat = g.ptr(a[2], kBf16, T, kLatent);
    void* rope = g.ptr(a[3], kBf16, T, kRope);
    void* st = g.opt(a[4], kI32, 1);
    if (!g.ok) Py_RETURN_NONE;
    return code(unlocked(f_read, static_cast<uint8_t*>(kv->data_ptr()), kv->size(0) * kv->size(1),
                       static_cast<int32_t*>(slot->data_ptr()), T, static_cast<uint16_t*>(lat),
                       static_cast<uint16_t*>(rope), static_cast<uint32_t*>(st), g.stream()));
  });
}

// Elements off .. off + len - 1 of a contiguous tensor, on the same storage (six
// narrow() calls through the dispatcher take 4 us, as long as the rest).
at::Tensor part(const at::Tensor& all, int64_t off, int64_t len) {
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(), all.dtype());
  t.unsafeGetTensorImpl()->set_storage_offset(off);
  t.unsafeGetTensorImpl()->set_sizes_contiguous({len});
  return t;
}

// block_tables(cached, new, table, free, begin, n_pages, page_size, T_cap, status)
// -> the six outputs, parts of one allocation
PyObject* block_tables(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args g;
    if (n != 9) Py_RETURN_NONE;
    const at::Tensor* cached = g.tensor(a[0], kI32, 1);
    const at::Tensor* table = g.tensor(a[2], kI32, 2);
    const at::Tensor* free_pages = g.tensor(a[3], kI32, 1);
    if (!g.ok) Py_RETURN_NONE;
    const int64_t B = cached->size(0), max_blocks = table->size(1);
    void* fresh = g.ptr(a[1], kI32, B);
    void* begin = g.ptr(a[4], kI32, 1);
    const int64_t n_pages = g.integer(a[5]), page_size = g.integer(a[6]), T = g.integer(a[7]);
    void* st = g.opt(a[8], kI32, 1);
    if (!g.ok || table->size(0) != B || T < 0 || T >= (int64_t(1) << 30) || !fits_int(B) || !fits_int(max_blocks) ||
        !fits_int(page_size))
      Py_RETURN_NONE;
    const at::Tensor all = at::empty({3 * T + 2 * B + 2}, g.options(kI32));
    int32_t* p = static_cast<int32_t*>(all.data_ptr());
    const int64_t len[6] = {T, T, T, B + 1, B, 1};
    int64_t off[6];
    for (int64_t i = 0, at = 0; i < 6; at += len[i++]) off[i] = at;
    const int rc = unlocked(f_tables, static_cast<int32_t*>(cached->data_ptr()), static_cast<int32_t*>(fresh), static_cast<int>(B),
                            static_cast<int32_t*>(table->data_ptr()), static_cast<int>(max_blocks),
                            static_cast<int32_t*>(free_pages->data_ptr()), free_pages->size(0), static_cast<int32_t*>(begin),
                            n_pages, static_cast<int>(page_size), T, p + off[0], p + off[1], p + off[2], p + off[3],
                            p + off[4], p + off[5], static_cast<uint32_t*>(st), g.stream());
    if (rc != 0) return code(rc);
    PyObject* out = PyTuple_New(6);
    if (!out) return nullptr;
    for (int i = 0; i < 6; ++i) {
      PyObject* o = THPVariable_Wrap(part(all, off[i], len[i]));
      if (!o) {
        Py_DECREF(out);
        return nullptr;
      }
      PyTuple_SET_ITEM(out, i, o);
    }
    return out;
  });
}

// prepare(fp8, q, k, position, inv_freq, k_out, k_scale, slot_map, q_norm,
// q_weight, q_bias, k_norm, k_weight, k_bias, eps, interleaved, q_out,
// q_scale, status) -> 0 or code; norms as numbers, bf16 or uint8 rows
PyObject* prepare(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args g;
    if (n != 19) Py_RETURN_NONE;
    const bool fp8 = g.integer(a[0]) != 0;
    const at::Tensor* q = g.tensor(a[1], kBf16, 3);
    const at::Tensor* freq = g.tensor(a[4], kF32, 1);
    if (!g.ok || !THPVariable_CheckExact(a[5])) Py_RETURN_NONE;
    const int64_t T = q->size(0), H = q->size(1), d = q->size(2);
    const int64_t k_dim = THPVariable_Unpack(a[5]).dim();
    const at::Tensor* k_out = g.tensor(a[5], fp8 ? kU8 : kBf16, k_dim);
    if (!g.ok || k_dim < 2 || k_out->size(k_dim - 1) != d || d == 0 || !fits_int(H) || !fits_int(2 * freq->size(0)))
      Py_RETURN_NONE;
    const int64_t slots = k_out->numel() / d;
    void* k = g.ptr(a[2], kBf16, T, d);
    void* pos = g.ptr(a[3], kI32, T);
    void* slot = g.opt(a[7], kI32, T);
    const int qn = static_cast<int>(g.integer(a[8])), kn = static_cast<int>(g.integer(a[11]));
    void *qw = g.opt(a[9], kF32, d), *qb = g.opt(a[10], kF32, d), *kw = g.opt(a[12], kF32, d), *kb = g.opt(a[13], kF32, d);
    if (!PyFloat_CheckExact(a[14]) || !PyBool_Check(a[15])) Py_RETURN_NONE;
    const float eps = static_cast<float>(PyFloat_AS_DOUBLE(a[14]));
    const int inter = a[15] == Py_True;
    void* q_out = g.ptr(a[16], fp8 ? kU8 : kBf16, T, H, d);
    void* st = g.opt(a[18], kI32, 1);
    auto F = [](void* x) { return static_cast<const float*>(x); };
    if (fp8) {
      const at::Tensor* ks = g.ok ? g.tensor(a[6], kF32, k_dim - 1) : nullptr;
      void* qs = g.ptr(a[17], kF32, T, H);
      if (!g.ok || ks->numel() != slots) Py_RETURN_NONE;
      for (int64_t i = 0; i + 1 < k_dim; ++i)
        if (ks->size(i) != k_out->size(i)) Py_RETURN_NONE;
      return code(unlocked(f_prepare8, static_cast<uint16_t*>(q->data_ptr()), static_cast<uint16_t*>(k), static_cast<int32_t*>(pos),
                             F(freq->data_ptr()), static_cast<int>(2 * freq->size(0)), T, static_cast<int>(H),
                             static_cast<int>(d), qn, F(qw), F(qb), kn, F(kw), F(kb), eps, inter,
                             static_cast<int32_t*>(slot), slots, static_cast<uint8_t*>(q_out), static_cast<float*>(qs),
                             static_cast<uint8_t*>(k_out->data_ptr()), static_cast<float*>(ks->data_ptr()),
                             static_cast<uint32_t*>(st), g.stream()));
    }
    if (!g.ok) Py_RETURN_NONE;
    return code(unlocked(f_prepare, static_cast<uint16_t*>(q->data_ptr()), static_cast<uint16_t*>(k), static_cast<int32_t*>(pos),
                          F(freq->data_ptr()), static_cast<int>(2 * freq->size(0)), T, static_cast<int>(H),
                          static_cast<int>(d), qn, F(qw), F(qb), kn, F(kw), F(kb), eps, inter,
                          static_cast<int32_t*>(slot), slots, static_cast<uint16_t*>(q_out),
                          static_cast<uint16_t*>(k_out->data_ptr()), static_cast<uint32_t*>(st), g.stream()));
  });
}

// attend(q, kv_pages, block_table, idx, scale, row_seq, out, lse, workspace,
// status) -> (out, lse) or code; out, lse and workspace may be None
PyObject* attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args g;
    if (n != 10) Py_RETURN_NONE;
    const at::Tensor* q = g.tensor(a[0], kBf16, 3);
    const at::Tensor* kv = g.tensor(a[1], kU8, 3);
    const at::Tensor* table = g.tensor(a[2], kI32, 2);
    const at::Tensor* idx = g.tensor(a[3], kI32, 2);
    if (!g.ok || kv->size(2) != DSA_KV4_ENTRY_BYTES || q->size(2) != kLatent + kRope || !PyFloat_CheckExact(a[4]))
      Py_RETURN_NONE;
    const int64_t T = q->size(0), H = q->size(1), m = idx->size(1), B = table->size(0), blocks = table->size(1);
    if (idx->size(0) != T || !fits_int(H) || !fits_int(m) || !fits_int(B) || !fits_int(blocks) || !fits_int(kv->size(1)))
      Py_RETURN_NONE;
    void* seq = g.opt(a[5], kI32, T);
    void* st = g.opt(a[9], kI32, 1);
    if (a[6] != Py_None) g.ptr(a[6], kBf16, T, H, kLatent);
    if (a[7] != Py_None) g.ptr(a[7], kF32, T, H);
    if (a[8] != Py_None) g.tensor(a[8], kU8, 1);
    if (!g.ok) Py_RETURN_NONE;
    at::Tensor out = a[6] != Py_None ? THPVariable_Unpack(a[6]) : at::empty({T, H, kLatent}, g.options(kBf16));
    at::Tensor lse = a[7] != Py_None ? THPVariable_Unpack(a[7]) : at::empty({T, H}, g.options(kF32));
    at::Tensor ws;
    if (a[8] != Py_None) {
      ws = THPVariable_Unpack(a[8]);
    } else {
      const size_t need = f_attend_ws(T, static_cast<int>(H), static_cast<int>(m));
      ws = at::empty({static_cast<int64_t>(need < 256 ? 256 : need)}, g.options(kU8));
    }
    const int rc = unlocked(f_attend, static_cast<uint16_t*>(q->data_ptr()), static_cast<uint8_t*>(kv->data_ptr()), kv->size(0),
                            static_cast<int>(kv->size(1)), static_cast<int32_t*>(table->data_ptr()), static_cast<int>(B),
                            static_cast<int>(blocks), static_cast<int32_t*>(seq), static_cast<int32_t*>(idx->data_ptr()), T,
                            static_cast<int>(H), static_cast<int>(m), static_cast<float>(PyFloat_AS_DOUBLE(a[4])),
                            static_cast<uint16_t*>(out.data_ptr()), static_cast<float*>(lse.data_ptr()), ws.data_ptr(),
                            static_cast<size_t>(ws.numel()), static_cast<uint32_t*>(st), g.stream());
    if (rc != 0) return code(rc);
    PyObject* o = a[6] != Py_None ? Py_NewRef(a[6]) : THPVariable_Wrap(out);
    PyObject* l = a[7] != Py_None ? Py_NewRef(a[7]) : THPVariable_Wrap(lse);
    PyObject* r = o && l ? PyTuple_Pack(2, o, l) : nullptr;
    Py_XDECREF(o);
    Py_XDECREF(l);
    return r;
  });
}

// bind(address of each entry point, in the order below)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void* v[7];
  if (n != 7) {
    PyErr_SetString(PyExc_TypeError, "bind takes seven addresses");
    return nullptr;
  }
  for (int i = 0; i < 7; ++i) {
    v[i] = PyLong_AsVoidPtr(a[i]);
    if (!v[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null entry point");
      return nullptr;
    }
  }
  f_tables = reinterpret_cast<decltype(f_tables)>(v[0]);
  f_prepare = reinterpret_cast<decltype(f_prepare)>(v[1]);
  f_prepare8 = reinterpret_cast<decltype(f_prepare8)>(v[2]);
  f_write = reinterpret_cast<decltype(f_write)>(v[3]);
  f_read = reinterpret_cast<decltype(f_read)>(v[4]);
  f_attend = reinterpret_cast<decltype(f_attend)>(v[5]);
  f_attend_ws = reinterpret_cast<decltype(f_attend_ws)>(v[6]);
  Py_RETURN_NONE;
}

#define FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(bind),    FAST(kv4_write), FAST(kv4_read), FAST(block_tables),
                         FAST(prepare), FAST(attend),    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serve_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serve_binding() { return PyModule_Create(&module); }
