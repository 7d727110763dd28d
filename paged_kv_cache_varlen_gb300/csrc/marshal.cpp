// marshal.cpp -- Python module `_marshal`: argument marshalling of the calls
// that a serving loop makes once a layer and step on small tensors (the rotary
// cache write and the cache-budget calls). It checks torch tensors as
// binding.py does, takes their pointers and calls libpkv; in Python the same
// checks took 7 to 15 us a call, more than the kernels of a small step.
// It computes nothing and keeps nothing.
#include <ATen/Context.h>
#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/impl/TorchDispatchModeTLS.h>
#include <c10/cuda/CUDAStream.h>
#include <cuda_runtime.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdlib>
#include <stdexcept>
#include <string>

#include "../../include/pkv.h"

namespace {

PyObject* g_error = nullptr;  // binding.PkvError

// A Python exception to raise: the type and its message.
struct Refused {
  PyObject* type;
  std::string text;
};

std::string shape_text(at::IntArrayRef s) {
  std::string t = "[";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + "]";
}

const char* type_name(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kFloat: return "torch.float32";
    case at::kDouble: return "torch.float64";
    case at::kInt: return "torch.int32";
    default: return c10::toString(t);
  }
}

// The call's device: that of its first tensor.
struct Call {
  int device = -1;

  const at::Tensor& any(PyObject* o, const char* name, at::ScalarType type, int64_t ndim) {
    if (!THPVariable_Check(o))
      throw Refused{PyExc_TypeError, std::string(name) + " must be a torch.Tensor"};
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda()) throw Refused{PyExc_ValueError, std::string(name) + " must be a CUDA tensor"};
    if (device < 0) device = t.get_device();
    if (t.get_device() != device)
      throw Refused{PyExc_ValueError, std::string(name) + " is on another device (cuda:" +
                                          std::to_string(t.get_device()) +
                                          ") than the first tensor"};
    if (t.scalar_type() != type)
      throw Refused{PyExc_TypeError, std::string(name) + " must be " + type_name(type) + ", got " +
                                         type_name(t.scalar_type())};
    if (t.dim() != ndim)
      throw Refused{PyExc_ValueError, std::string(name) + " must have " + std::to_string(ndim) +
                                          " dims, got shape " + shape_text(t.sizes())};
    return t;
  }
  const at::Tensor& dense(PyObject* o, const char* name, at::ScalarType type, int64_t ndim) {
    const at::Tensor& t = any(o, name, type, ndim);
    if (!t.is_contiguous())
      throw Refused{PyExc_ValueError, std::string(name) + " must be contiguous"};
    return t;
  }
  const at::Tensor& kv_pool(PyObject* o) {
    const at::Tensor& t = dense(o, "kv_pool", at::kBFloat16, 5);
    if (t.size(0) != 2)
      throw Refused{PyExc_ValueError,
                    "kv_pool must be [2, num_blocks, block_size, num_kv_heads, head_dim], got " +
                        shape_text(t.sizes())};
    return t;
  }
  // [tokens, heads, head_dim] bf16, a token's heads contiguous; the distance
  // between tokens goes to *stride.
  const at::Tensor& rows(PyObject* o, const char* name, int64_t tokens, int64_t heads,
                         int64_t head_dim, int64_t* stride) {
    const at::Tensor& t = any(o, name, at::kBFloat16, 3);
    if (t.size(0) != tokens || t.size(1) != heads || t.size(2) != head_dim)
      throw Refused{PyExc_ValueError, std::string(name) + " must be " +
                                          shape_text({tokens, heads, head_dim}) + ", got " +
                                          shape_text(t.sizes())};
    if ((head_dim > 1 && t.stride(2) != 1) || (heads > 1 && t.stride(1) != head_dim))
      throw Refused{PyExc_ValueError,
                    std::string(name) + ": the heads of a token must be contiguous, got strides " +
                        shape_text(t.strides())};
    *stride = tokens > 1 ? t.stride(0) : heads * head_dim;
    return t;
  }
  int32_t* ints(PyObject* o, const char* name, int64_t length) {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = dense(o, name, at::kInt, 1);
    if (length >= 0 && t.size(0) != length)
      throw Refused{PyExc_ValueError, std::string(name) + " must have one entry per request"};
    return static_cast<int32_t*>(t.data_ptr());
  }
};

template <class T = void>
T* ptr(const at::Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}

// torch.empty of bf16. Its way through the dispatcher (0.7 us a call) is left out
// where nothing there would act: no dispatch mode, and no filling of new memory
// in deterministic mode.
at::Tensor new_output(at::IntArrayRef shape, c10::Device device) {
  const at::Context& context = at::globalContext();
  if (c10::impl::dispatch_mode_enabled() ||
      (context.deterministicAlgorithms() && context.deterministicFillUninitializedMemory()))
    return at::empty(shape, at::TensorOptions(device).dtype(at::kBFloat16));
  return at::Tensor(at::detail::empty_cuda(shape, at::kBFloat16, device, std::nullopt));
}

int32_t small(int64_t v) {
  if (v > INT32_MAX || v < INT32_MIN)
    throw Refused{PyExc_ValueError, "a size does not fit 32 bits"};
  return (int32_t)v;
}
int64_t to_int(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused{nullptr, ""};
  return v;
}
float to_float(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused{nullptr, ""};
  return (float)v;
}

// `call(stream)` with the tensors' device current, on the given stream (an
// integer handle) or torch's current one; raises PkvError on a status. The
// interpreter lock is given up meanwhile, as ctypes and torch do: a launch waits
// while the stream's queue is full. (`call` touches no Python object.)
template <class F>
void run(const char* what, int device, PyObject* stream, F call) {
  void* s = nullptr;
  if (stream == Py_None)
    s = c10::cuda::getCurrentCUDAStream(device).stream();
  else
    s = reinterpret_cast<void*>(static_cast<uintptr_t>(PyLong_AsUnsignedLongLong(stream)));
  if (PyErr_Occurred()) throw Refused{nullptr, ""};
  // Takes the lock again, whatever `call` throws. (At the interpreter's end that
  // unwinds a daemon thread, which a destructor must let through.)
  struct Unlocked {
    PyThreadState* state = PyEval_SaveThread();
    ~Unlocked() noexcept(false) { PyEval_RestoreThread(state); }
  };
  struct Device {  // puts the current device back, whatever `call` throws
    int now = -1, used = -1;
    ~Device() {
      if (used >= 0 && now != used) cudaSetDevice(now);
    }
  };
  pkv_status st = PKV_ERR_CUDA;
  {
    Unlocked unlocked;
    Device current;
    if (cudaGetDevice(&current.now) == cudaSuccess &&
        (current.now == device || cudaSetDevice(device) == cudaSuccess)) {
      current.used = device;
      st = call(s);
    }
  }
  if (st == PKV_OK) return;
  const std::string text = std::string(what) + ": " + pkv_status_string(st) + " (status " +
                           std::to_string(st) + ")";
  PyObject* e = PyObject_CallFunction(g_error, "si", text.c_str(), (int)st);
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Refused{nullptr, ""};
}

// Runs `body`, turning what it throws into a Python exception.
template <class F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, F body) {
  if (got != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", want, got);
    return nullptr;
  }
  try {
    return body();
  } catch (const Refused& r) {
    if (r.type) PyErr_SetString(r.type, r.text.c_str());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// q, kv_pool, k_new, v_new, positions, slot_mapping, inv_freq, interleaved,
// factor, q_out, dev_status, stream
PyObject* rope_kv_cache_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> PyObject* {
    Call c;
    const at::Tensor& pool = c.kv_pool(a[1]);
    const at::Tensor& positions = c.dense(a[4], "positions", at::kInt, 1);
    const at::Tensor& slots = c.dense(a[5], "slot_mapping", at::kInt, 1);
    const at::Tensor& inv_freq = c.dense(a[6], "inv_freq", at::kDouble, 1);
    const int64_t t = slots.size(0), hkv = pool.size(3), d = pool.size(4);
    if (positions.size(0) != t)
      throw Refused{PyExc_ValueError, "positions and slot_mapping differ in length"};
    const int64_t h = c.any(a[0], "q", at::kBFloat16, 3).size(1);
    int64_t qs, ks, vs;
    const at::Tensor& q = c.rows(a[0], "q", t, h, d, &qs);
    const at::Tensor& k = c.rows(a[2], "k_new", t, hkv, d, &ks);
    const at::Tensor& v = c.rows(a[3], "v_new", t, hkv, d, &vs);
    at::Tensor made;
    if (a[9] == Py_None) {
      made = new_output({t, h, d}, q.device());
    } else if (c.dense(a[9], "q_out", at::kBFloat16, 3).sizes() != q.sizes()) {
      throw Refused{PyExc_ValueError, "q_out must have the shape of q"};
    }
    const at::Tensor& out = a[9] == Py_None ? made : THPVariable_Unpack(a[9]);
    int32_t* status = c.ints(a[10], "dev_status", -1);
    const int interleaved = PyObject_IsTrue(a[7]);
    if (interleaved < 0) throw Refused{nullptr, ""};
    const float factor = to_float(a[8]);
    run("rope_kv_cache_write", c.device, a[11], [&](void* stream) {
      return pkv_rope_kv_cache_write(
          ptr(out), ptr(pool), ptr(q), ptr(k), ptr(v), qs, ks, vs, ptr<int32_t>(positions),
          ptr<int32_t>(slots), ptr<double>(inv_freq), factor, interleaved, small(t), small(h),
          small(hkv), small(d), small(2 * inv_freq.size(0)), small(pool.size(1)),
          small(pool.size(2)), status, stream);
    });
    if (a[9] == Py_None) return THPVariable_Wrap(made);
    Py_INCREF(a[9]);
    return a[9];
  });
}

// q, kv_pool, lse, block_table, cu_seqlens, seq_lens, max_query_len,
// max_seq_len, weights, out, weight_rows, prior_lens, decay, scale (None:
// 1 / sqrt(head_dim)), dev_status, stream
PyObject* attention_key_weights(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 16, [&]() -> PyObject* {
    Call c;
    const at::Tensor& pool = c.kv_pool(a[1]);
    const at::Tensor& q = c.dense(a[0], "q", at::kBFloat16, 3);
    const at::Tensor& lse = c.dense(a[2], "lse", at::kFloat, 2);
    const at::Tensor& table = c.dense(a[3], "block_table", at::kInt, 2);
    const at::Tensor& cu = c.dense(a[4], "cu_seqlens", at::kInt, 1);
    const at::Tensor& lens = c.dense(a[5], "seq_lens", at::kInt, 1);
    const at::Tensor& weights = c.dense(a[8], "weights", at::kFloat, 3);
    const int64_t t = q.size(0), h = q.size(1), d = q.size(2), hkv = pool.size(3);
    const int64_t b = lens.size(0);
    if (pool.size(4) != d) throw Refused{PyExc_ValueError, "q and kv_pool head_dim differ"};
    if (lse.size(0) != t || lse.size(1) != h)
      throw Refused{PyExc_ValueError, "lse must be [num_tokens, num_heads]"};
    if (cu.size(0) != b + 1 || table.size(0) != b)
      throw Refused{PyExc_ValueError, "cu_seqlens must be [B+1] and block_table [B, max_blocks]"};
    if (weights.size(1) != hkv)
      throw Refused{PyExc_ValueError, "weights must be [rows, num_kv_heads, row_len]"};
    PyObject* result = a[9] == Py_None ? a[8] : a[9];
    const at::Tensor& out = c.dense(result, "out", at::kFloat, 3);
    if (out.sizes() != weights.sizes())
      throw Refused{PyExc_ValueError, "out must have the shape of weights"};
    const int32_t* rows = c.ints(a[10], "weight_rows", b);
    const int32_t* prior = c.ints(a[11], "prior_lens", b);
    int32_t* status = c.ints(a[14], "dev_status", -1);
    const int32_t max_q = small(to_int(a[6])), max_len = small(to_int(a[7]));
    const float decay = to_float(a[12]);
    const float scale = a[13] == Py_None ? (float)(1.0 / std::sqrt((double)d)) : to_float(a[13]);
    run("attention_key_weights", c.device, a[15], [&](void* stream) {
      return pkv_attention_key_weights(
          ptr<float>(out), ptr<float>(weights), ptr(q), ptr(pool), ptr<float>(lse),
          ptr<int32_t>(table), small(table.size(1)), ptr<int32_t>(cu), ptr<int32_t>(lens), prior,
          rows, small(weights.size(0)), small(weights.size(2)), small(b), small(t), max_q, max_len,
          small(h), small(hkv), small(d), small(pool.size(2)), small(pool.size(1)), scale, decay,
          status, stream);
    });
    Py_INCREF(result);
    return result;
  });
}

// weights, seq_lens, keep_lens, max_seq_len, max_keep_len, num_sink,
// num_recent, weight_rows, kept, weights_out, dev_status, stream
PyObject* evict_select(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> PyObject* {
    Call c;
    const at::Tensor& weights = c.dense(a[0], "weights", at::kFloat, 3);
    const at::Tensor& lens = c.dense(a[1], "seq_lens", at::kInt, 1);
    const at::Tensor& keep = c.dense(a[2], "keep_lens", at::kInt, 1);
    const at::Tensor& kept = c.dense(a[8], "kept", at::kInt, 3);
    const int64_t b = lens.size(0), hkv = weights.size(1);
    const int32_t max_len = small(to_int(a[3])), max_keep = small(to_int(a[4]));
    if (keep.size(0) != b)
      throw Refused{PyExc_ValueError, "seq_lens and keep_lens differ in length"};
    if (kept.size(0) != b || kept.size(1) != hkv || kept.size(2) != max_keep)
      throw Refused{PyExc_ValueError, "kept must be [num_seqs, num_kv_heads, max_keep_len]"};
    float* out = nullptr;
    if (a[9] != Py_None) {
      const at::Tensor& o = c.dense(a[9], "weights_out", at::kFloat, 3);
      if (o.sizes() != weights.sizes())
        throw Refused{PyExc_ValueError, "weights_out must have the shape of weights"};
      out = ptr<float>(o);
    }
    const int32_t* rows = c.ints(a[7], "weight_rows", b);
    int32_t* status = c.ints(a[10], "dev_status", -1);
    const int32_t sink = small(to_int(a[5])), recent = small(to_int(a[6]));
    run("evict_select", c.device, a[11], [&](void* stream) {
      return pkv_evict_select(ptr<int32_t>(kept), out, ptr<float>(weights), ptr<int32_t>(lens),
                              ptr<int32_t>(keep), rows, small(weights.size(0)),
                              small(weights.size(2)), small(b), small(hkv), max_len, max_keep, sink,
                              recent, status, stream);
    });
    Py_RETURN_NONE;
  });
}

// kv_pool, src_table, dst_table, kept, keep_lens, dev_status, stream
PyObject* evict_compact(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&]() -> PyObject* {
    Call c;
    const at::Tensor& pool = c.kv_pool(a[0]);
    const at::Tensor& src = c.dense(a[1], "src_table", at::kInt, 2);
    const at::Tensor& dst = c.dense(a[2], "dst_table", at::kInt, 2);
    const at::Tensor& kept = c.dense(a[3], "kept", at::kInt, 3);
    const at::Tensor& keep = c.dense(a[4], "keep_lens", at::kInt, 1);
    const int64_t b = keep.size(0), hkv = pool.size(3);
    if (kept.size(0) != b || kept.size(1) != hkv)
      throw Refused{PyExc_ValueError, "kept must be [num_seqs, num_kv_heads, max_keep_len]"};
    if (src.size(0) != b || dst.size(0) != b)
      throw Refused{PyExc_ValueError, "src_table and dst_table must have one row per request"};
    int32_t* status = c.ints(a[5], "dev_status", -1);
    run("evict_compact", c.device, a[6], [&](void* stream) {
      return pkv_evict_compact(ptr(pool), ptr<int32_t>(src), small(src.size(1)), ptr<int32_t>(dst),
                               small(dst.size(1)), ptr<int32_t>(kept), small(kept.size(2)),
                               ptr<int32_t>(keep), small(b), small(hkv), small(pool.size(4)),
                               small(pool.size(2)), small(pool.size(1)), status, stream);
    });
    Py_RETURN_NONE;
  });
}

// Whether PKV_DEBUG_CHECKS is set to 1 now (os.environ writes through to the C
// environment; asking there takes 0.05 us, os.environ.get of a missing name 0.6).
PyObject* debug_checks(PyObject*, PyObject*) {
  const char* v = std::getenv("PKV_DEBUG_CHECKS");
  return PyBool_FromLong(v && v[0] == '1' && v[1] == '\0');
}

// set_error(PkvError)
PyObject* set_error(PyObject*, PyObject* type) {
  Py_INCREF(type);
  Py_XDECREF(g_error);
  g_error = type;
  Py_RETURN_NONE;
}

#define PKV_FAST(f) \
  { #f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr }
PyMethodDef kMethods[] = {PKV_FAST(rope_kv_cache_write),
                          PKV_FAST(attention_key_weights),
                          PKV_FAST(evict_select),
                          PKV_FAST(evict_compact),
                          {"debug_checks", debug_checks, METH_NOARGS, nullptr},
                          {"set_error", set_error, METH_O, nullptr},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&kModule); }
