// Python binding of the paged-serving operators: checks devices and strides,
// describes torch tensors, allocates outputs and calls the C ABI
// (include/fia.h) on the current stream.  A server calls these operators every
// few microseconds for every layer, so the marshalling is compiled: a ctypes
// call of eight tensors cost 26 us of host time, this one a fifth.
// _paged.py holds the public functions; their arguments arrive here by position.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <optional>
#include <string>

#include "../../include/fia.h"

namespace {

PyObject* g_error = nullptr;   // FIAError(status, detail)

struct Raised {};              // a Python exception is set

[[noreturn]] void raise(PyObject* type, const std::string& what) {
  PyErr_SetString(type, what.c_str());
  throw Raised();
}

void check(fia_status s) {
  if (s == FIA_OK) return;
  PyObject* e = PyObject_CallFunction(g_error, "is", int(s), fia_last_error());
  if (e != nullptr) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Raised();
}

// Positional arguments of one call, and the device all its tensors share.
struct Call {
  PyObject* const* args;
  Py_ssize_t n;
  std::optional<c10::Device> device;

  Call(PyObject* const* a, Py_ssize_t have, Py_ssize_t want) : args(a), n(have) {
    if (have != want) raise(PyExc_TypeError, "wrong number of arguments");
  }
  bool none(int i) const { return args[i] == Py_None; }
  // The i-th argument as a tensor on the call's device.
  const at::Tensor& tensor(int i, const char* name) {
    if (!THPVariable_Check(args[i])) raise(PyExc_TypeError, std::string(name) + " must be a tensor");
    const at::Tensor& t = THPVariable_Unpack(args[i]);
    if (!t.is_cuda()) raise(PyExc_ValueError, "fia kernels take CUDA tensors");
    if (!device) device = t.device();
    if (t.device() != *device) raise(PyExc_ValueError, "tensors must be on one device");
    return t;
  }
  int64_t integer(int i) const {
    const long long v = PyLong_AsLongLong(args[i]);
    if (v == -1 && PyErr_Occurred()) throw Raised();
    return v;
  }
  double real(int i) const {
    const double v = PyFloat_AsDouble(args[i]);
    if (v == -1.0 && PyErr_Occurred()) throw Raised();
    return v;
  }
  bool truth(int i) const {
    const int v = PyObject_IsTrue(args[i]);
    if (v < 0) throw Raised();
    return v != 0;
  }
};

int dtype_code(at::ScalarType t) {
  switch (t) {
    case at::kHalf: return FIA_DTYPE_F16;
    case at::kBFloat16: return FIA_DTYPE_BF16;
    case at::kFloat: return FIA_DTYPE_F32;
    case at::kInt: return FIA_DTYPE_I32;
    case at::kLong: return FIA_DTYPE_I64;
    case at::kByte: return FIA_DTYPE_U8;
    case at::kBool: return FIA_DTYPE_BOOL;
    case at::kChar: return FIA_DTYPE_I8;
    case at::kFloat8_e4m3fn: return FIA_DTYPE_F8E4M3;
    default: raise(PyExc_TypeError, std::string("unsupported dtype ") + c10::toString(t));
  }
}

fia_tensor describe(const at::Tensor& t, const char* name) {
  fia_tensor d;
  std::memset(&d, 0, sizeof(d));
  if (t.dim() > 5) raise(PyExc_ValueError, std::string(name) + " has more than 5 dims");
  d.data = t.numel() > 0 ? t.data_ptr() : nullptr;
  d.dtype = dtype_code(t.scalar_type());
  d.ndim = int32_t(t.dim());
  for (int i = 0; i < d.ndim; ++i) d.shape[i] = t.size(i);
  return d;
}

// Descriptor of a contiguous argument; None gives an absent one.
struct Desc {
  fia_tensor d;
  bool here = false;
  Desc() { std::memset(&d, 0, sizeof(d)); }
  Desc(Call& c, int i, const char* name) : Desc() {
    if (c.none(i)) return;
    set(c.tensor(i, name), name);
  }
  void set(const at::Tensor& t, const char* name) {
    if (!t.is_contiguous()) raise(PyExc_ValueError, std::string(name) + " must be contiguous");
    d = describe(t, name);
    here = true;
  }
  const fia_tensor* ptr() const { return here ? &d : nullptr; }
};

// (the allocator called directly: through torch's dispatcher an output costs
// twice as much host time)
at::Tensor empty(at::IntArrayRef shape, at::ScalarType t, c10::Device dev) {
  return at::detail::empty_cuda(shape, t, dev, std::nullopt);
}

// An output argument: the caller's, or a new one of this shape and type.
at::Tensor output(Call& c, int i, const char* name, at::IntArrayRef shape, at::ScalarType t) {
  return c.none(i) ? empty(shape, t, *c.device) : c.tensor(i, name);
}

PyObject* wrap(const at::Tensor& t) { return THPVariable_Wrap(t); }

PyObject* pair(const at::Tensor& a, const std::optional<at::Tensor>& b) {
  PyObject* x = wrap(a);
  PyObject* y = b ? wrap(*b) : Py_NewRef(Py_None);
  PyObject* r = x != nullptr && y != nullptr ? PyTuple_Pack(2, x, y) : nullptr;
  Py_XDECREF(x);
  Py_XDECREF(y);
  return r;
}

// Query, lse and the parameters that every attention call starts with:
//   num_heads, num_key_value_heads, scale_value, input_layout, pre_tokens,
//   block_size, softmax_lse_flag, out, softmax_lse  from argument i on.
struct Attention {
  fia_params prm;
  at::Tensor out;
  std::optional<at::Tensor> lse;
  Desc out_d, lse_d;

  Attention(Call& c, const at::Tensor& q, int i) {
    fia_params_init(&prm);
    prm.num_heads = c.integer(i);
    prm.num_key_value_heads = c.integer(i + 1);
    prm.scale_value = c.real(i + 2);
    prm.input_layout = PyUnicode_AsUTF8(c.args[i + 3]);
    if (prm.input_layout == nullptr) throw Raised();
    prm.pre_tokens = c.integer(i + 4);
    prm.block_size = c.integer(i + 5);
    prm.softmax_lse_flag = c.truth(i + 6) ? 1 : 0;
    out = c.none(i + 7) ? empty(q.sizes(), q.scalar_type(), *c.device) : c.tensor(i + 7, "out");
    out_d.set(out, "out");
    if (!c.none(i + 8)) {
      lse = c.tensor(i + 8, "softmax_lse");
    } else if (prm.softmax_lse_flag != 0 && q.dim() >= 3) {
      const int64_t H = prm.num_heads;
      if (std::strcmp(prm.input_layout, "TND") == 0)
        lse = empty({q.size(0), H, 1}, at::kFloat, *c.device);
      else
        lse = empty({q.size(0), H, std::strcmp(prm.input_layout, "BNSD") == 0 ? q.size(2) : q.size(1), 1}, at::kFloat,
                    *c.device);
    }
    if (lse) lse_d.set(*lse, "softmax_lse");
  }
  PyObject* result() const { return pair(out, lse); }
};

template <typename F>
PyObject* guarded(F&& f) {
  try {
    return f();
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

void* stream_of(const Call& c) { return c10::cuda::getCurrentCUDAStream(c.device->index()).stream(); }

// context_lens, new_lens, free_blocks, block_table, block_size, num_tokens,
// slot_mapping, kv_lens, cu_new_lens, num_blocks
PyObject* block_table_append(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call c(args, n, 10);
    Desc ctx(c, 0, "context_lens"), add(c, 1, "new_lens"), free(c, 2, "free_blocks"), table(c, 3, "block_table");
    if (!c.device) raise(PyExc_TypeError, "context_lens must be a tensor");
    const at::Tensor& lens = c.tensor(0, "context_lens");
    const int64_t bs = c.integer(4), tokens = c.integer(5);
    if (tokens < 0) raise(PyExc_ValueError, "num_tokens must be 0 or more");
    const at::cuda::CUDAGuard on(*c.device);
    at::Tensor o[4] = {output(c, 6, "slot_mapping", {tokens}, at::kInt), output(c, 7, "kv_lens", lens.sizes(), at::kInt),
                       output(c, 8, "cu_new_lens", lens.sizes(), at::kInt), output(c, 9, "num_blocks", {1}, at::kInt)};
    if (o[0].dim() != 1 || o[0].size(0) != tokens) raise(PyExc_ValueError, "slot_mapping must have num_tokens entries");
    static const char* const names[4] = {"slot_mapping", "kv_lens", "cu_new_lens", "num_blocks"};
    Desc d[4];
    for (int i = 0; i < 4; ++i) d[i].set(o[i], names[i]);
    check(fia_block_table_append(ctx.ptr(), add.ptr(), free.ptr(), bs, table.ptr(), d[0].ptr(), d[1].ptr(), d[2].ptr(),
                                 d[3].ptr(), stream_of(c)));
    PyObject* r = PyTuple_New(4);
    if (r == nullptr) return nullptr;
    for (int i = 0; i < 4; ++i) {
      PyObject* x = wrap(o[i]);
      if (x == nullptr) {
        Py_DECREF(r);
        return nullptr;
      }
      PyTuple_SET_ITEM(r, i, x);
    }
    return r;
  });
}

// Elements between the tokens of a (T, N, D) tensor whose heads and columns
// are contiguous.
int64_t token_stride(const at::Tensor& t, const char* name) {
  if (t.dim() != 3) raise(PyExc_ValueError, std::string(name) + " must be (T, KV_N, D)");
  const int64_t N = t.size(1), D = t.size(2);
  if ((D > 1 && t.stride(2) != 1) || (N > 1 && t.stride(1) != D))
    raise(PyExc_ValueError, std::string(name) + ": the heads and columns of a token must be contiguous");
  if (t.size(0) < 2) return N * D;
  // (the C entry reads a stride of 0 as "contiguous")
  if (t.stride(0) < N * D) raise(PyExc_ValueError, std::string(name) + ": tokens must not share memory");
  return t.stride(0);
}

// key, value, key_cache, value_cache, slot_mapping
PyObject* cache_write(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call c(args, n, 5);
    const at::Tensor& key = c.tensor(0, "key");
    const fia_tensor k = describe(key, "key");
    const int64_t ks = token_stride(key, "key");
    fia_tensor v;
    int64_t vs = 0;
    const bool two = !c.none(1);
    if (two) {
      const at::Tensor& value = c.tensor(1, "value");
      v = describe(value, "value");
      vs = token_stride(value, "value");
    }
    Desc kc(c, 2, "key_cache"), vc(c, 3, "value_cache"), slots(c, 4, "slot_mapping");
    const at::cuda::CUDAGuard on(*c.device);
    check(fia_cache_write(&k, ks, two ? &v : nullptr, vs, kc.ptr(), vc.ptr(), slots.ptr(), stream_of(c)));
    return PyTuple_Pack(2, args[2], args[3]);
  });
}

// query, key, value, actual_seq_kvlen, block_table, sink_tokens, attention...
PyObject* decode_window(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call c(args, n, 15);
    const at::Tensor& q = c.tensor(0, "query");
    const at::cuda::CUDAGuard on(*c.device);
    Desc qd(c, 0, "query"), k(c, 1, "key"), v(c, 2, "value"), lens(c, 3, "actual_seq_kvlen"), table(c, 4, "block_table");
    const int64_t sink = c.integer(5);
    Attention a(c, q, 6);
    check(fia_decode_window(qd.ptr(), k.ptr(), v.ptr(), table.ptr(), lens.ptr(), &a.prm, sink, a.out_d.ptr(),
                            a.lse_d.ptr(), stream_of(c)));
    return a.result();
  });
}

// The workspace argument, or a new one of `bytes` (asked for when needed).
template <typename F>
at::Tensor workspace(Call& c, int i, F&& bytes) {
  if (c.none(i)) return empty({int64_t(bytes())}, at::kByte, *c.device);
  const at::Tensor& t = c.tensor(i, "workspace");
  if (!t.is_contiguous()) raise(PyExc_ValueError, "workspace must be contiguous");
  return t;
}

// query, key, value, actual_seq_qlen, actual_seq_kvlen, block_table,
// sink_tokens, attention..., workspace
PyObject* prefill_window(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call c(args, n, 17);
    const at::Tensor& q = c.tensor(0, "query");
    const at::cuda::CUDAGuard on(*c.device);
    Desc qd(c, 0, "query"), k(c, 1, "key"), v(c, 2, "value"), ql(c, 3, "actual_seq_qlen"), kl(c, 4, "actual_seq_kvlen"),
        table(c, 5, "block_table");
    const int64_t sink = c.integer(6);
    Attention a(c, q, 7);
    const at::Tensor ws = workspace(c, 16, [&] {
      size_t need = 0;
      check(fia_prefill_window_get_workspace_size(qd.ptr(), k.ptr(), v.ptr(), table.ptr(), ql.ptr(), kl.ptr(), &a.prm, sink,
                                                  a.out_d.ptr(), a.lse_d.ptr(), &need));
      return need;
    });
    check(fia_prefill_window(qd.ptr(), k.ptr(), v.ptr(), table.ptr(), ql.ptr(), kl.ptr(), &a.prm, sink, a.out_d.ptr(),
                             a.lse_d.ptr(), ws.data_ptr(), size_t(ws.nbytes()), stream_of(c)));
    return a.result();
  });
}

// query, key_cache, value_cache, actual_seq_kvlen, block_table,
// shared_prefix_len, attention..., workspace
PyObject* decode_shared_prefix(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Call c(args, n, 16);
    const at::Tensor& q = c.tensor(0, "query");
    const at::cuda::CUDAGuard on(*c.device);
    Desc qd(c, 0, "query"), k(c, 1, "key_cache"), v(c, 2, "value_cache"), kl(c, 3, "actual_seq_kvlen"),
        table(c, 4, "block_table");
    const int64_t prefix = c.integer(5);
    Attention a(c, q, 6);
    const at::Tensor ws = workspace(c, 15, [&] {
      size_t need = 0;
      check(fia_decode_shared_prefix_get_workspace_size(qd.ptr(), k.ptr(), v.ptr(), table.ptr(), kl.ptr(), &a.prm, prefix,
                                                        a.out_d.ptr(), a.lse_d.ptr(), &need));
      return need;
    });
    check(fia_decode_shared_prefix(qd.ptr(), k.ptr(), v.ptr(), table.ptr(), kl.ptr(), &a.prm, prefix, a.out_d.ptr(),
                                   a.lse_d.ptr(), ws.data_ptr(), size_t(ws.nbytes()), stream_of(c)));
    return a.result();
  });
}

// The exception class that a failing call raises.
PyObject* set_error(PyObject*, PyObject* cls) {
  Py_XSETREF(g_error, Py_NewRef(cls));
  Py_RETURN_NONE;
}

#define FIA_FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {FIA_FAST(block_table_append), FIA_FAST(cache_write), FIA_FAST(decode_window),
                           FIA_FAST(prefill_window), FIA_FAST(decode_shared_prefix), {"set_error", set_error, METH_O, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_fia_paged", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fia_paged() { return PyModule_Create(&g_module); }
