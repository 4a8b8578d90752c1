// torch_calls.cpp -- the short way from PyTorch tensors to the library's rotation, 8-bit cache and its attention.
//
// A call of these takes microseconds on the GPU when it serves a few tokens, and from Python, through the checks of torch_ops.py,
// PyTorch's allocations and ctypes, 15 - 20 us on a Grace core.  The functions here take the arguments as torch_ops.py gets them and,
// where every one is of the form that the library reads as it is, allocate the outputs and the workspace, call the library under
// torch_ops.py's lock and return the outputs (a decoding step's rotation 8 instead of 19 us, its attention 9 instead of 22).  In every other case, and for
// every refusal, they return None and have done nothing: torch_ops.py then copies, checks and explains.
#include <Python.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <ATen/core/grad_mode.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <array>
#include <exception>

#include "domino.h"

namespace {

constexpr int64_t kD = 128;
constexpr int kMaxDevices = 64;

// The library's functions, as addresses from the one that is loaded, its handles, and the lock that they are used under.
struct Library {
  decltype(&domino_qk_rotary_fwd) rotary_fwd;
  decltype(&domino_qk_rotary_bwd) rotary_bwd;
  decltype(&domino_qk_rotary_bwd_workspace_size) rotary_bwd_size;
  decltype(&domino_cache_write) cache_write;
  decltype(&domino_cache_read) cache_read;
  decltype(&domino_attn_cached_fwd) attn;
  decltype(&domino_attn_cached_workspace_size) attn_size;
} library;
domino_handle handles[kMaxDevices];
PyObject *lock_acquire, *lock_release;

const at::Tensor* tensor(PyObject* o) { return THPVariable_CheckExact(o) ? &THPVariable_Unpack(o) : nullptr; }

// What a call has looked at so far: `ok` while all of it is of the plain form.
struct Look {
  bool ok = true;
  int device = -1;
  int64_t tokens = -1;

  bool fail() { return ok = false; }

  // [tokens, heads, 128] bf16, heads one after the other, tokens at one 16-byte aligned stride.
  struct Heads {
    const uint16_t* p = nullptr;
    int64_t heads = 0, ld = 0;
  };
  Heads heads(PyObject* o, bool differentiable = false) {
    Heads h;
    const at::Tensor* x = tensor(o);
    if (!ok || !x || !on_device(*x) || x->scalar_type() != at::kBFloat16 || x->dim() != 3 || (differentiable && x->requires_grad())) {
      fail();
      return h;
    }
    const auto n = x->sizes(), s = x->strides();
    if (tokens < 0) tokens = n[0];
    const auto at = reinterpret_cast<uintptr_t>(x->data_ptr());
    h.heads = n[1];
    h.ld = n[0] <= 1 ? h.heads * kD : s[0];
    if (n[0] != tokens || n[2] != kD || h.heads < 1 || s[2] != 1 || (s[1] != kD && h.heads != 1) || h.ld < h.heads * kD || h.ld % 8 || at & 15) fail();
    h.p = reinterpret_cast<const uint16_t*>(at);
    return h;
  }
  // A contiguous vector of n values (any number: n < 0).
  template <class T>
  const T* vec(PyObject* o, at::ScalarType type, int64_t n, uintptr_t align = 0) {
    const at::Tensor* x = tensor(o);
    if (!ok || !x || !on_device(*x) || x->scalar_type() != type || x->dim() != 1 || (n >= 0 && x->size(0) != n) || !x->is_contiguous() ||
        reinterpret_cast<uintptr_t>(x->data_ptr()) & align) {
      fail();
      return nullptr;
    }
    return static_cast<const T*>(x->data_ptr());
  }
  bool on_device(const at::Tensor& x) {
    if (!x.is_cuda() || x.layout() != at::kStrided) return false;
    const int d = x.get_device();
    if (device < 0) {
      device = d;
      return d >= 0 && d < kMaxDevices && handles[d] && c10::cuda::current_device() == d;
    }
    return d == device;
  }
};

// Positions, frequencies, weights and the like: positions, frequencies, q_weight, k_weight, layout, eps, amplitude.
struct Rotation {
  const int32_t* positions = nullptr;
  const double* frequencies = nullptr;
  const uint16_t *wq = nullptr, *wk = nullptr;
  int32_t rot = 0, layout = 0;
  float eps = 0, amplitude = 0;

  Rotation(Look& look, PyObject* const* a, int64_t hq, int64_t hkv, bool differentiable = false) {
    if (!look.ok) return;
    if ((a[0] == Py_None) != (a[1] == Py_None)) {
      look.fail();
      return;
    }
    if (a[0] != Py_None) {
      positions = look.vec<int32_t>(a[0], at::kInt, look.tokens);
      frequencies = look.vec<double>(a[1], at::kDouble, -1);
      if (look.ok) {
        const int64_t n = tensor(a[1])->size(0);
        if (n > kD / 2 || n % 8) look.fail();
        rot = static_cast<int32_t>(2 * n);
      }
    }
    const bool q = a[2] != Py_None, k = a[3] != Py_None;
    if (q || k) {
      if (q != (hq > 0) || k != (hkv > 0)) look.fail();
      if (q) wq = look.vec<uint16_t>(a[2], at::kBFloat16, kD, 15);
      if (k) wk = look.vec<uint16_t>(a[3], at::kBFloat16, kD, 15);
      if (differentiable && look.ok && ((q && tensor(a[2])->requires_grad()) || (k && tensor(a[3])->requires_grad()))) look.fail();
    }
    const long code = PyLong_CheckExact(a[4]) ? PyLong_AsLong(a[4]) : -1;
    if (code != DOMINO_ROTARY_HALF && code != DOMINO_ROTARY_INTERLEAVED) look.fail();
    layout = static_cast<int32_t>(code);
    eps = number(look, a[5]);
    amplitude = number(look, a[6]);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      look.fail();
    }
  }
  static float number(Look& look, PyObject* o) {
    if (!PyFloat_CheckExact(o) && !PyLong_CheckExact(o)) look.fail();
    return look.ok ? static_cast<float>(PyFloat_AsDouble(o)) : 0.0f;
  }
};

// The cache's four tensors, contiguous.
struct Cache {
  const uint8_t *k8 = nullptr, *v8 = nullptr, *k_exp = nullptr, *v_exp = nullptr;
  int64_t rows = 0, heads = 0;

  Cache(Look& look, PyObject* o) {
    if (!look.ok || !PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 4) {
      look.fail();
      return;
    }
    const at::Tensor* x[4];
    for (int i = 0; i < 4; ++i) {
      x[i] = tensor(PyTuple_GET_ITEM(o, i));
      if (!x[i] || !look.on_device(*x[i]) || !x[i]->is_contiguous() || x[i]->scalar_type() != (i < 2 ? at::kFloat8_e4m3fn : at::kByte) ||
          x[i]->dim() != (i < 2 ? 3 : 2)) {
        look.fail();
        return;
      }
    }
    rows = x[0]->size(0);
    heads = x[0]->size(1);
    for (int i = 0; i < 2; ++i) {
      const at::Tensor &c = *x[i], &e = *x[i + 2];
      if (c.size(0) != rows || c.size(1) != heads || c.size(2) != kD || e.size(0) != heads || e.size(1) != rows || heads < 1 ||
          reinterpret_cast<uintptr_t>(c.data_ptr()) & 15)
        look.fail();
    }
    k8 = static_cast<const uint8_t*>(x[0]->data_ptr());
    v8 = static_cast<const uint8_t*>(x[1]->data_ptr());
    k_exp = static_cast<const uint8_t*>(x[2]->data_ptr());
    v_exp = static_cast<const uint8_t*>(x[3]->data_ptr());
  }
};

at::Tensor made(at::IntArrayRef size, at::ScalarType type, int device) {
  return at::empty(size, at::TensorOptions().dtype(type).device(at::Device(at::kCUDA, static_cast<at::DeviceIndex>(device))));
}
uint16_t* bits(const at::Tensor& x) { return x.defined() ? static_cast<uint16_t*>(x.data_ptr()) : nullptr; }

// A workspace on the stream, given back when the call is enqueued: it is reused in the stream's order.
struct Scratch {
  void* p = nullptr;
  Scratch(size_t size, cudaStream_t st) {
    if (size) p = c10::cuda::CUDACachingAllocator::raw_alloc_with_stream(size, st);
  }
  ~Scratch() {
    if (p) c10::cuda::CUDACachingAllocator::raw_delete(p);
  }
  Scratch(const Scratch&) = delete;
  Scratch& operator=(const Scratch&) = delete;
};

// Runs `work(handle, stream)`, which allocates and calls the library, without the interpreter's lock and under torch_ops.py's; false
// where another thread has that one, or the library refuses.
template <class Work>
bool enqueue(int device, Work&& work) {
  PyObject* const got = PyObject_CallOneArg(lock_acquire, Py_False);
  if (!got) throw python_error();
  const bool mine = got == Py_True;
  Py_DECREF(got);
  if (!mine) return false;
  domino_status status = DOMINO_OK;
  std::exception_ptr thrown;
  PyThreadState* const state = PyEval_SaveThread();
  try {
    status = work(handles[device], c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream());
  } catch (...) {
    thrown = std::current_exception();
  }
  PyEval_RestoreThread(state);
  PyObject* const given = PyObject_CallNoArgs(lock_release);
  if (thrown) {
    Py_XDECREF(given);
    std::rethrow_exception(thrown);
  }
  if (!given) throw python_error();
  Py_DECREF(given);
  return status == DOMINO_OK;
}

PyObject* wrapped(const at::Tensor& x) {
  if (x.defined()) return THPVariable_Wrap(x);
  Py_RETURN_NONE;
}
template <size_t N>
PyObject* wrapped(const std::array<at::Tensor, N>& x) {
  PyObject* const t = PyTuple_New(N);
  if (!t) throw python_error();
  for (size_t i = 0; i < N; ++i) {
    PyObject* const o = wrapped(x[i]);
    if (!o) {
      Py_DECREF(t);
      throw python_error();
    }
    PyTuple_SET_ITEM(t, i, o);
  }
  return t;
}

// ---- the functions; their arguments by position, all of them

// q, k, then a rotation's -> (q', k')
PyObject* qk_rotary_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 9) Py_RETURN_NONE;
  Look look;
  const auto q = look.heads(a[0]);
  Look::Heads k;
  if (a[1] != Py_None) k = look.heads(a[1]);
  const Rotation r(look, a + 2, q.heads, k.heads);
  if (!look.ok) Py_RETURN_NONE;
  std::array<at::Tensor, 2> y;
  const bool done = enqueue(look.device, [&](domino_handle h, cudaStream_t st) {
    y[0] = made({look.tokens, q.heads, kD}, at::kBFloat16, look.device);
    if (k.p || k.heads) y[1] = made({look.tokens, k.heads, kD}, at::kBFloat16, look.device);
    return library.rotary_fwd(h, q.p, q.ld, k.p, k.ld, r.positions, r.frequencies, r.rot, r.layout, r.amplitude, r.wq, r.wk, r.eps, bits(y[0]),
                              q.heads * kD, bits(y[1]), k.heads * kD, look.tokens, static_cast<int32_t>(q.heads),
                              static_cast<int32_t>(k.heads), st);
  });
  if (!done) Py_RETURN_NONE;
  return wrapped(y);
  END_HANDLE_TH_ERRORS
}

// gq, gk, q, k, then a rotation's -> (gq, gk, gq_weight, gk_weight)
PyObject* qk_rotary_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 11) Py_RETURN_NONE;
  Look look;
  const auto gq = look.heads(a[0]);
  Look::Heads gk, q, k;
  if (a[1] != Py_None) gk = look.heads(a[1]);
  const Rotation r(look, a + 4, gq.heads, gk.heads);
  const bool norm = r.wq != nullptr;
  if (norm) {
    q = look.heads(a[2]);
    if ((a[3] != Py_None) != (gk.heads > 0)) look.fail();
    if (look.ok && gk.heads) k = look.heads(a[3]);
    if (q.heads != gq.heads || k.heads != gk.heads) look.fail();
  }
  if (!look.ok) Py_RETURN_NONE;
  std::array<at::Tensor, 4> g;
  const bool done = enqueue(look.device, [&](domino_handle h, cudaStream_t st) {
    const int32_t hq = static_cast<int32_t>(gq.heads), hkv = static_cast<int32_t>(gk.heads);
    g[0] = made({look.tokens, gq.heads, kD}, at::kBFloat16, look.device);
    if (hkv) g[1] = made({look.tokens, gk.heads, kD}, at::kBFloat16, look.device);
    size_t size = 0;
    if (norm) {
      g[2] = made({kD}, at::kFloat, look.device);
      if (hkv) g[3] = made({kD}, at::kFloat, look.device);
      const domino_status s = library.rotary_bwd_size(look.tokens, hq, hkv, &size);
      if (s != DOMINO_OK) return s;
    }
    const Scratch ws(size, st);
    return library.rotary_bwd(h, gq.p, gq.ld, gk.p, gk.ld, q.p, q.ld, k.p, k.ld, r.positions, r.frequencies, r.rot, r.layout, r.amplitude, r.wq,
                              r.wk, r.eps, bits(g[0]), gq.heads * kD, bits(g[1]), gk.heads * kD,
                              g[2].defined() ? static_cast<float*>(g[2].data_ptr()) : nullptr,
                              g[3].defined() ? static_cast<float*>(g[3].data_ptr()) : nullptr, 0, look.tokens, hq, hkv, ws.p, size, st);
  });
  if (!done) Py_RETURN_NONE;
  return wrapped(g);
  END_HANDLE_TH_ERRORS
}

// cache, rows, k, v, q, then a rotation's -> (q',), or (None,) without q
PyObject* cache_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 12) Py_RETURN_NONE;
  const bool grad = at::GradMode::is_enabled();
  Look look;
  const auto k = look.heads(a[2], grad), v = look.heads(a[3], grad);
  const Cache c(look, a[0]);
  const int32_t* rows = look.ok ? look.vec<int32_t>(a[1], at::kInt, look.tokens) : nullptr;
  Look::Heads q;
  if (a[4] != Py_None) q = look.heads(a[4], grad);
  const Rotation r(look, a + 5, q.heads, k.heads, grad);
  if (!look.ok || k.heads != c.heads || v.heads != c.heads) Py_RETURN_NONE;
  std::array<at::Tensor, 1> y;
  const bool done = enqueue(look.device, [&](domino_handle h, cudaStream_t st) {
    if (q.heads) y[0] = made({look.tokens, q.heads, kD}, at::kBFloat16, look.device);
    return library.cache_write(h, q.p, q.ld, k.p, k.ld, v.p, v.ld, r.positions, r.frequencies, r.rot, r.layout, r.amplitude, r.wq, r.wk, r.eps,
                               bits(y[0]), q.heads * kD, rows, const_cast<uint8_t*>(c.k8), const_cast<uint8_t*>(c.v8),
                               const_cast<uint8_t*>(c.k_exp), const_cast<uint8_t*>(c.v_exp), c.rows, c.rows, look.tokens,
                               static_cast<int32_t>(q.heads), static_cast<int32_t>(k.heads), st);
  });
  if (!done) Py_RETURN_NONE;
  return wrapped(y);
  END_HANDLE_TH_ERRORS
}

// cache, rows -> (k, v)
PyObject* cache_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 2) Py_RETURN_NONE;
  Look look;
  const int32_t* rows = look.vec<int32_t>(a[1], at::kInt, -1);
  const Cache c(look, a[0]);
  if (!look.ok) Py_RETURN_NONE;
  const int64_t tokens = tensor(a[1])->size(0);
  std::array<at::Tensor, 2> x;
  const bool done = enqueue(look.device, [&](domino_handle h, cudaStream_t st) {
    for (auto& y : x) y = made({tokens, c.heads, kD}, at::kBFloat16, look.device);
    return library.cache_read(h, c.k8, c.v8, c.k_exp, c.v_exp, c.rows, c.rows, rows, bits(x[0]), c.heads * kD, bits(x[1]), c.heads * kD, tokens,
                              static_cast<int32_t>(c.heads), st);
  });
  if (!done) Py_RETURN_NONE;
  return wrapped(x);
  END_HANDLE_TH_ERRORS
}

// q, cache, k_start, k_len, prefix, scale, return_lse -> (o, lse), or (o, None)
PyObject* cached_attention(PyObject*, PyObject* const* a, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  if (count != 7 || !PyFloat_CheckExact(a[5])) Py_RETURN_NONE;
  Look look;
  const at::Tensor* q = tensor(a[0]);
  if (!q || !look.on_device(*q) || q->scalar_type() != at::kBFloat16 || (q->dim() != 3 && q->dim() != 4) ||
      (q->requires_grad() && at::GradMode::is_enabled()))
    Py_RETURN_NONE;
  const Cache c(look, a[1]);
  if (!look.ok) Py_RETURN_NONE;
  const auto size = q->sizes(), s = q->strides();
  const bool several = q->dim() == 4;
  const int64_t n = size[0], t = several ? size[1] : 1, hq = size[several + 1];
  // one stride from token to token
  const int64_t step = t > 1 ? s[1] : s[0], ld = n * t <= 1 ? hq * kD : step;
  const auto at = reinterpret_cast<uintptr_t>(q->data_ptr());
  if (size[several + 2] != kD || hq < 1 || hq % c.heads || s[several + 2] != 1 || (s[several + 1] != kD && hq != 1) || (n > 1 && t > 1 && s[0] != t * s[1]) ||
      ld < hq * kD || ld % 8 || at & 15)
    Py_RETURN_NONE;
  const int32_t *start = look.vec<int32_t>(a[2], at::kInt, n), *len = look.vec<int32_t>(a[3], at::kInt, n),
                *prefix = a[4] != Py_None ? look.vec<int32_t>(a[4], at::kInt, 2) : nullptr;
  if (!look.ok) Py_RETURN_NONE;
  const float scale = static_cast<float>(PyFloat_AS_DOUBLE(a[5]));
  std::array<at::Tensor, 2> y;
  const bool done = enqueue(look.device, [&](domino_handle h, cudaStream_t st) {
    const int32_t heads = static_cast<int32_t>(hq), kv_heads = static_cast<int32_t>(c.heads);
    size_t bytes = 0;
    const domino_status refused = library.attn_size(n, t, heads, kv_heads, prefix != nullptr, &bytes);
    if (refused != DOMINO_OK) return refused;
    y[0] = made(size, at::kBFloat16, look.device);
    if (a[6] == Py_True) y[1] = made(size.slice(0, size.size() - 1), at::kFloat, look.device);
    const Scratch ws(bytes, st);
    return library.attn(h, reinterpret_cast<const uint16_t*>(at), ld, c.k8, c.v8, c.k_exp, c.v_exp, c.rows, c.rows, start, len, prefix, scale,
                        bits(y[0]), hq * kD, y[1].defined() ? static_cast<float*>(y[1].data_ptr()) : nullptr, n, t, heads, kv_heads, ws.p, bytes, st);
  });
  if (!done) Py_RETURN_NONE;
  return wrapped(y);
  END_HANDLE_TH_ERRORS
}

// The library's addresses in the order of Library, and the lock.
PyObject* use(PyObject*, PyObject* const* a, Py_ssize_t n) {
  constexpr Py_ssize_t kFunctions = sizeof(Library) / sizeof(void*);
  void* p[kFunctions];
  if (n != kFunctions + 1) {
    PyErr_SetString(PyExc_TypeError, "use: the library's functions and the lock");
    return nullptr;
  }
  for (Py_ssize_t i = 0; i < kFunctions; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  PyObject *acquire = PyObject_GetAttrString(a[kFunctions], "acquire"), *release = PyObject_GetAttrString(a[kFunctions], "release");
  if (!acquire || !release) {
    Py_XDECREF(acquire);
    Py_XDECREF(release);
    return nullptr;
  }
  memcpy(&library, p, sizeof(p));
  Py_XSETREF(lock_acquire, acquire);
  Py_XSETREF(lock_release, release);
  Py_RETURN_NONE;
}
// A device's handle.
PyObject* use_handle(PyObject*, PyObject* const* a, Py_ssize_t n) {
  const long device = n == 2 ? PyLong_AsLong(a[0]) : -1;
  void* h = n == 2 ? PyLong_AsVoidPtr(a[1]) : nullptr;
  if (PyErr_Occurred()) return nullptr;
  if (device >= 0 && device < kMaxDevices) handles[device] = static_cast<domino_handle>(h);
  Py_RETURN_NONE;
}

#define FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(qk_rotary_fwd), FAST(qk_rotary_bwd), FAST(cache_write), FAST(cache_read), FAST(cached_attention),
                         FAST(use),           FAST(use_handle),    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "torch_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// `built_for`: the PyTorch whose headers lay out the tensors that are read here.
PyMODINIT_FUNC PyInit_torch_calls() {
  PyObject* const m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "built_for", TORCH_VERSION) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
