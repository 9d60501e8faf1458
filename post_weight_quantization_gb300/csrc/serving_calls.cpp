// The serving operators' calls for the case that a decoding loop makes: tensors of the right kinds
// and shapes on the current device, work on the current stream. Each function takes its Python
// namesake's arguments, looks the tensors over, allocates what is missing and calls the library; it
// returns None, with nothing done, for any argument that is not plainly right. The caller then goes
// the long way, whose checks say what is wrong (or allow what is merely unusual).
//
// Why: attribute reads and ctypes cost the host more than a small call's kernels cost the GPU. Measured,
// the long way / this one, in us a call: 33 tokens of gptq_qk_norm_rope 20.2 / 6.2 (host alone 18 / 5),
// gptq_kv_append with gptq_kv_read 24.7 / 9.2, gptq_kv_attention over 331 tokens 21.9 / 10.2,
// gptq_adapter_linear of one token 24.5 / 12.3.
#include <Python.h>

#include <cmath>
#include <initializer_list>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include "gptq.h"

namespace {

constexpr int kBad = -1;

struct Decline {};                                         // thrown where an argument is not plainly right

long long integer(PyObject* o) {
  const long long v = PyLong_Check(o) ? PyLong_AsLongLong(o) : -1;
  if (!PyLong_Check(o) || (v == -1 && PyErr_Occurred())) throw Decline{};
  return v;
}
int small(PyObject* o) {
  const long long v = integer(o);
  if (v != (int)v) throw Decline{};
  return (int)v;
}
float real(PyObject* o) {
  if (!PyFloat_Check(o)) throw Decline{};
  return (float)PyFloat_AS_DOUBLE(o);
}
bool flag(PyObject* o) {
  if (o == Py_True) return true;
  if (o == Py_False) return false;
  throw Decline{};
}

int code_of(at::ScalarType t) {
  return t == at::kFloat ? GPTQ_F32 : t == at::kBFloat16 ? GPTQ_BF16 : t == at::kHalf ? GPTQ_F16 : kBad;
}

// The device of a call: that of its first tensor, which must be the current one.
struct Call {
  int dev;
  cudaStream_t stream;
  explicit Call(PyObject* first) {
    const at::Tensor& t = tensor(first);
    if (!t.is_cuda()) throw Decline{};
    dev = t.get_device();
    if (dev != c10::cuda::current_device()) throw Decline{};
    stream = c10::cuda::getCurrentCUDAStream(dev).stream();
  }
  static const at::Tensor& tensor(PyObject* o) {
    if (!THPVariable_Check(o)) throw Decline{};
    return THPVariable_Unpack(o);
  }
  const at::Tensor& on(PyObject* o) const {
    const at::Tensor& t = tensor(o);
    if (!t.is_cuda() || t.get_device() != dev) throw Decline{};
    return t;
  }
  // a contiguous tensor of this type and shape
  void* dense(PyObject* o, at::ScalarType type, std::initializer_list<int64_t> shape) const {
    const at::Tensor& t = on(o);
    if (t.scalar_type() != type || !t.sizes().equals(shape) || !t.is_contiguous()) throw Decline{};
    return t.data_ptr();
  }
  void* dense_or_null(PyObject* o, at::ScalarType type, std::initializer_list<int64_t> shape) const {
    return o == Py_None ? nullptr : dense(o, type, shape);
  }
  // a (tokens, heads, dim) tensor whose heads lie densely in a token's row; its token stride
  int64_t heads(const at::Tensor& t, int64_t tokens, int64_t n, int64_t dim) const {
    if (t.dim() != 3 || (tokens >= 0 && t.size(0) != tokens) || (n >= 0 && t.size(1) != n) || (dim >= 0 && t.size(2) != dim))
      throw Decline{};
    if (t.numel() && (t.stride(2) != 1 || (t.size(1) > 1 && t.stride(1) != t.size(2)))) throw Decline{};
    return t.size(0) > 1 ? t.stride(0) : t.size(1) * t.size(2);
  }
  // a (tokens, d) tensor of this type with unit column stride; its row stride
  static int64_t rows(const at::Tensor& t, at::ScalarType type, int64_t tokens, int64_t d) {
    if (t.scalar_type() != type || t.dim() != 2 || t.size(0) != tokens || t.size(1) != d || t.stride(1) != 1) throw Decline{};
    return tokens > 1 ? t.stride(0) : d;
  }
  at::Tensor make(std::initializer_list<int64_t> shape, at::ScalarType type) const {
    return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, dev));
  }
  // a workspace of `need` bytes: the caller's, or one of this call
  void* workspace(PyObject* o, size_t need, size_t& bytes, at::Tensor& own) const {
    if (o == Py_None) {
      bytes = need > 256 ? need : 256;
      own = make({(int64_t)bytes}, at::kByte);
      return own.data_ptr();
    }
    const at::Tensor& t = on(o);
    if (t.scalar_type() != at::kByte || !t.is_contiguous()) throw Decline{};
    bytes = (size_t)t.numel();
    return t.data_ptr();
  }
};

// The library's call without the interpreter's lock: a launch waits while the stream's queue is full,
// and other threads go on meanwhile, as they do in the long way. About 0.3 us a call. (`f` touches no Python
// object; the arguments' tensors are held by the caller.)
template <typename F>
void call(F&& f) {
  PyThreadState* state = PyEval_SaveThread();
  const gptq_status st = f();
  PyEval_RestoreThread(state);
  if (st != GPTQ_OK) throw Decline{};                      // the long way reports it
}

template <int N, typename F>
PyObject* guarded(Py_ssize_t n, F&& f) {
  if (n != N) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return f();
  } catch (...) {                                          // among them the allocator's: the long way raises its own
    PyErr_Clear();
  }
  Py_RETURN_NONE;
}

PyObject* back(PyObject* given, const at::Tensor& t) {
  if (given == Py_None) return THPVariable_Wrap(t);
  Py_INCREF(given);
  return given;
}

PyObject* three(PyObject* x, PyObject* y, PyObject* z) {
  PyObject* all = x && y && z ? PyTuple_Pack(3, x, y, z) : nullptr;
  Py_XDECREF(x);
  Py_XDECREF(y);
  Py_XDECREF(z);
  return all;
}

// qweight, scales, zeros, d, bits, group_size, X, m, A, B, ids, alpha, Y, out_bf16, ws -> Y
PyObject* adapter_linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded<15>(n, [&]() -> PyObject* {
    const Call c(a[6]);
    const at::Tensor& X = c.on(a[6]);
    const int64_t d = integer(a[3]), m = integer(a[7]);
    const int bits = small(a[4]), gs = small(a[5]);
    if (X.scalar_type() != at::kBFloat16 || X.dim() != 2 || X.size(1) != d || X.stride(1) != 1) throw Decline{};
    if (d <= 0 || m <= 0 || (d * bits) % 32 || !(gs == -1 || (gs > 0 && d % gs == 0))) throw Decline{};
    const int64_t T = X.size(0), G = gs == -1 ? 1 : d / gs;
    auto* qw = c.dense(a[0], at::kInt, {m, d * bits / 32});
    auto* sc = c.dense(a[1], at::kFloat, {m, G});
    auto* ze = c.dense(a[2], at::kFloat, {m, G});
    int64_t na = 0;
    int rank = 8;
    void *A = nullptr, *B = nullptr, *ids = nullptr, *alpha = nullptr;
    if (a[8] != Py_None) {
      const at::Tensor& t = c.on(a[8]);
      if (t.dim() != 3) throw Decline{};
      na = t.size(0);
      rank = (int)t.size(1);
      A = c.dense(a[8], at::kBFloat16, {na, rank, d});
      B = c.dense(a[9], at::kBFloat16, {na, m, rank});
      ids = c.dense(a[10], at::kInt, {T});
      alpha = c.dense_or_null(a[11], at::kFloat, {na});
    } else if (a[9] != Py_None || a[10] != Py_None || a[11] != Py_None) {
      throw Decline{};
    }
    const at::ScalarType yt = flag(a[13]) ? at::kBFloat16 : at::kFloat;
    const at::Tensor Y = a[12] == Py_None ? c.make({T, m}, yt) : c.on(a[12]);
    if (Y.scalar_type() != yt || Y.dim() != 2 || Y.size(0) != T || Y.size(1) != m || Y.stride(1) != 1) throw Decline{};
    at::Tensor own;
    size_t bytes = 0;
    void* ws = c.workspace(a[14], gptq_adapter_workspace_size(m, d, bits, gs, T, rank), bytes, own);
    call([&] {
      return gptq_adapter_linear((const uint32_t*)qw, (const float*)sc, (const float*)ze, m, d, bits, gs,
                                 (const uint16_t*)X.data_ptr(), T, T > 1 ? X.stride(0) : d, (const uint16_t*)A, (const uint16_t*)B,
                                 (const float*)alpha, na, rank, (const int32_t*)ids, Y.data_ptr(),
                                 yt == at::kBFloat16 ? GPTQ_BF16 : GPTQ_F32, T > 1 ? Y.stride(0) : m, ws, bytes, c.stream);
    });
    return back(a[12], Y);
  });
}

// Q, K, positions, cos, sin, wq, wk, eps, interleaved, Q_out, K_out, out_dtype -> (Q_out, K_out)
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded<12>(n, [&]() -> PyObject* {
    const Call c(a[0]);
    const at::Tensor& Q = c.on(a[0]);
    const at::ScalarType in = Q.scalar_type();
    const int64_t ldq = c.heads(Q, -1, -1, -1), T = Q.size(0), hq = Q.size(1), dim = Q.size(2);
    at::ScalarType out = in;
    if (a[11] != Py_None) {
      if (!THPDtype_Check(a[11])) throw Decline{};
      out = reinterpret_cast<THPDtype*>(a[11])->scalar_type;
    } else if (a[9] != Py_None) {
      out = c.on(a[9]).scalar_type();
    }
    if (code_of(in) == kBad || code_of(out) == kBad) throw Decline{};
    const at::Tensor Qo = a[9] == Py_None ? c.make({T, hq, dim}, out) : c.on(a[9]);
    if (Qo.scalar_type() != out) throw Decline{};
    const int64_t ldqo = c.heads(Qo, T, hq, dim);
    int64_t hk = 0, ldk = 0, ldko = 0;
    void* K = nullptr;
    at::Tensor Ko;
    if (a[1] != Py_None) {
      const at::Tensor& t = c.on(a[1]);
      if (t.scalar_type() != in) throw Decline{};
      ldk = c.heads(t, T, -1, dim);
      hk = t.size(1);
      K = t.data_ptr();
      Ko = a[10] == Py_None ? c.make({T, hk, dim}, out) : c.on(a[10]);
      if (Ko.scalar_type() != out) throw Decline{};
      ldko = c.heads(Ko, T, hk, dim);
    } else if (a[6] != Py_None || a[10] != Py_None) {
      throw Decline{};
    }
    int64_t n_pos = 0, rot = 0;
    void *pos = nullptr, *cs = nullptr, *sn = nullptr;
    if (a[3] != Py_None) {
      const at::Tensor& t = c.on(a[3]);
      if (t.dim() != 2) throw Decline{};
      n_pos = t.size(0);
      rot = 2 * t.size(1);
      cs = c.dense(a[3], at::kFloat, {n_pos, rot / 2});
      sn = c.dense(a[4], at::kFloat, {n_pos, rot / 2});
      pos = c.dense(a[2], at::kInt, {T});
    } else if (a[2] != Py_None || a[4] != Py_None) {
      throw Decline{};
    }
    void* wq = c.dense_or_null(a[5], at::kFloat, {dim});
    void* wk = c.dense_or_null(a[6], at::kFloat, {dim});
    const float eps = real(a[7]);
    const bool interleaved = flag(a[8]);
    call([&] {
      return gptq_qk_norm_rope(Q.data_ptr(), K, code_of(in), T, (int)hq, (int)hk, (int)dim, ldq, ldk, (const float*)wq,
                               (const float*)wk, eps, (const float*)cs, (const float*)sn, n_pos, (int)rot, interleaved,
                               (const int32_t*)pos, Qo.data_ptr(), Ko.defined() ? Ko.data_ptr() : nullptr, code_of(out),
                               ldqo, ldko, c.stream);
    });
    PyObject* q = back(a[9], Qo);
    PyObject* k = Ko.defined() ? back(a[10], Ko) : Py_NewRef(Py_None);
    PyObject* both = q && k ? PyTuple_Pack(2, q, k) : nullptr;
    Py_XDECREF(q);
    Py_XDECREF(k);
    return both;
  });
}

// X, R, w, eps, R_out, Y, out_dtype, scale -> (Y, R_out, scale)
PyObject* add_rms_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded<8>(n, [&]() -> PyObject* {
    const Call c(a[0]);
    const at::Tensor& X = c.on(a[0]);
    const at::ScalarType in = X.scalar_type();
    if (code_of(in) == kBad || X.dim() != 2) throw Decline{};
    const int64_t T = X.size(0), d = X.size(1), ldx = Call::rows(X, in, T, d);
    at::ScalarType out = in;
    if (a[6] != Py_None) {
      if (!THPDtype_Check(a[6])) throw Decline{};
      out = reinterpret_cast<THPDtype*>(a[6])->scalar_type;
    } else if (a[5] != Py_None) {
      out = c.on(a[5]).scalar_type();
    }
    const bool bytes = out == at::kFloat8_e4m3fn;
    if (!bytes && code_of(out) == kBad) throw Decline{};
    int64_t ldr = 0, ldro = 0;
    void* R = nullptr;
    at::Tensor Ro, scale;
    if (a[1] != Py_None) {
      const at::Tensor& t = c.on(a[1]);
      ldr = Call::rows(t, in, T, d);
      R = t.data_ptr();
      Ro = a[4] == Py_None ? c.make({T, d}, in) : c.on(a[4]);
      ldro = Call::rows(Ro, in, T, d);
    } else if (a[4] != Py_None) {
      throw Decline{};
    }
    void* w = c.dense_or_null(a[2], at::kFloat, {d});
    const float eps = real(a[3]);
    const at::Tensor Y = a[5] == Py_None ? c.make({T, d}, out) : c.on(a[5]);
    const int64_t ldy = Call::rows(Y, out, T, d);
    if (bytes) {
      if (a[7] != Py_None) c.dense(a[7], at::kFloat, {T});
      scale = a[7] == Py_None ? c.make({T}, at::kFloat) : c.on(a[7]);
    } else if (a[7] != Py_None) {
      throw Decline{};
    }
    call([&] {
      return gptq_add_rms_norm(X.data_ptr(), R, code_of(in), T, d, ldx, ldr, (const float*)w, eps,
                               R ? Ro.data_ptr() : nullptr, ldro, Y.data_ptr(), bytes ? GPTQ_E4M3 : code_of(out), ldy,
                               bytes ? (float*)scale.data_ptr() : nullptr, c.stream);
    });
    return three(back(a[5], Y), Ro.defined() ? back(a[4], Ro) : Py_NewRef(Py_None),
                 bytes ? back(a[7], scale) : Py_NewRef(Py_None));
  });
}

// qweight, scales, zeros, d, bits, group_size, X, m, x_scale, bias, act, mul, residual, A, B, ids, alpha, Y, out_bf16, ws -> Y
PyObject* linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded<20>(n, [&]() -> PyObject* {
    const Call c(a[6]);
    const at::Tensor& X = c.on(a[6]);
    const int64_t d = integer(a[3]), m = integer(a[7]);
    const int bits = small(a[4]), gs = small(a[5]), act = small(a[10]);
    const bool bytes = X.scalar_type() == at::kFloat8_e4m3fn;
    if (!(bytes || X.scalar_type() == at::kBFloat16) || X.dim() != 2) throw Decline{};
    if (d <= 0 || m <= 0 || (d * bits) % 32 || !(gs == -1 || (gs > 0 && d % gs == 0))) throw Decline{};
    const int64_t T = X.size(0), G = gs == -1 ? 1 : d / gs, ldx = Call::rows(X, X.scalar_type(), T, d);
    auto* qw = c.dense(a[0], at::kInt, {m, d * bits / 32});
    auto* sc = c.dense(a[1], at::kFloat, {m, G});
    auto* ze = c.dense(a[2], at::kFloat, {m, G});
    if (bytes != (a[8] != Py_None)) throw Decline{};
    void* xs = c.dense_or_null(a[8], at::kFloat, {T});
    void* bias = c.dense_or_null(a[9], at::kFloat, {m});
    const at::ScalarType yt = flag(a[18]) ? at::kBFloat16 : at::kFloat;
    const void* more[2] = {nullptr, nullptr};
    int64_t ld[2] = {0, 0};
    for (int i = 0; i < 2; ++i) {
      if (a[11 + i] == Py_None) continue;
      const at::Tensor& t = c.on(a[11 + i]);
      ld[i] = Call::rows(t, yt, T, m);
      more[i] = t.data_ptr();
    }
    int64_t na = 0;
    int rank = 0;
    void *A = nullptr, *B = nullptr, *ids = nullptr, *alpha = nullptr;
    if (a[13] != Py_None) {
      const at::Tensor& t = c.on(a[13]);
      if (t.dim() != 3 || bytes) throw Decline{};
      na = t.size(0);
      rank = (int)t.size(1);
      A = c.dense(a[13], at::kBFloat16, {na, rank, d});
      B = c.dense(a[14], at::kBFloat16, {na, m, rank});
      ids = c.dense(a[15], at::kInt, {T});
      alpha = c.dense_or_null(a[16], at::kFloat, {na});
    } else if (a[14] != Py_None || a[15] != Py_None || a[16] != Py_None) {
      throw Decline{};
    }
    if (na == 0) {                                         // none to choose from: none
      rank = 0;
      A = B = ids = alpha = nullptr;
    }
    const at::Tensor Y = a[17] == Py_None ? c.make({T, m}, yt) : c.on(a[17]);
    const int64_t ldy = Call::rows(Y, yt, T, m);
    const int xt = bytes ? GPTQ_E4M3 : GPTQ_BF16;
    at::Tensor own;
    size_t size = 0;
    void* ws = c.workspace(a[19], gptq_linear_workspace_size(m, d, bits, gs, T, xt, rank), size, own);
    call([&] {
      return gptq_linear((const uint32_t*)qw, (const float*)sc, (const float*)ze, m, d, bits, gs, X.data_ptr(), xt, T, ldx,
                         (const float*)xs, (const uint16_t*)A, (const uint16_t*)B, (const float*)alpha, na, rank,
                         (const int32_t*)ids, (const float*)bias, act, more[0], ld[0], more[1], ld[1], Y.data_ptr(),
                         yt == at::kBFloat16 ? GPTQ_BF16 : GPTQ_F32, ldy, ws, size, c.stream);
    });
    return back(a[17], Y);
  });
}

// logits, u, temperature, top_k, top_p, min_p, tokens, logprob -> (tokens, logprob)
PyObject* sample(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded<8>(n, [&]() -> PyObject* {
    const Call c(a[0]);
    const at::Tensor& L = c.on(a[0]);
    const at::ScalarType type = L.scalar_type();
    if (code_of(type) == kBad || L.dim() != 2) throw Decline{};
    const int64_t rows = L.size(0), vocab = L.size(1), ld = Call::rows(L, type, rows, vocab);
    void* u = c.dense(a[1], at::kFloat, {rows});
    void* temperature = c.dense_or_null(a[2], at::kFloat, {rows});
    void* top_k = c.dense_or_null(a[3], at::kInt, {rows});
    void* top_p = c.dense_or_null(a[4], at::kFloat, {rows});
    void* min_p = c.dense_or_null(a[5], at::kFloat, {rows});
    if (a[6] != Py_None) c.dense(a[6], at::kInt, {rows});
    if (a[7] != Py_None) c.dense(a[7], at::kFloat, {rows});
    const at::Tensor tokens = a[6] == Py_None ? c.make({rows}, at::kInt) : c.on(a[6]);
    const at::Tensor logprob = a[7] == Py_None ? c.make({rows}, at::kFloat) : c.on(a[7]);
    call([&] {
      return gptq_sample(L.data_ptr(), code_of(type), rows, vocab, ld, (const float*)u, (const float*)temperature,
                         (const int32_t*)top_k, (const float*)top_p, (const float*)min_p, (int32_t*)tokens.data_ptr(),
                         (float*)logprob.data_ptr(), c.stream);
    });
    PyObject *t = back(a[6], tokens), *l = back(a[7], logprob);
    PyObject* both = t && l ? PyTuple_Pack(2, t, l) : nullptr;
    Py_XDECREF(t);
    Py_XDECREF(l);
    return both;
  });
}

struct Pool {
  void* data;
  int64_t pages;
  int page, heads, dim;
  Pool(const Call& c, PyObject* pool, PyObject* page_size, PyObject* n_kv_heads, PyObject* head_dim)
      : page(small(page_size)), heads(small(n_kv_heads)), dim(small(head_dim)) {
    const at::Tensor& t = c.on(pool);
    if (t.dim() != 3) throw Decline{};
    pages = t.size(0);
    data = c.dense(pool, at::kByte, {pages, heads, (int64_t)page * (dim + 8)});
  }
};

// pool, page_size, n_kv_heads, head_dim, K, V, slots -> True
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded<7>(n, [&]() -> PyObject* {
    const Call c(a[4]);
    const Pool p(c, a[0], a[1], a[2], a[3]);
    const at::Tensor &K = c.on(a[4]), &V = c.on(a[5]);
    const at::ScalarType type = K.scalar_type();
    if (code_of(type) == kBad || V.scalar_type() != type) throw Decline{};
    const int64_t ldk = c.heads(K, -1, p.heads, p.dim), T = K.size(0), ldv = c.heads(V, T, p.heads, p.dim);
    void* slots = c.dense(a[6], at::kLong, {T});
    call([&] {
      return gptq_kv_append(K.data_ptr(), V.data_ptr(), code_of(type), T, p.heads, p.dim, ldk, ldv, (const int64_t*)slots,
                            p.data, p.pages, p.page, c.stream);
    });
    Py_RETURN_TRUE;
  });
}

// pool, page_size, n_kv_heads, head_dim, slots, dtype, K, V -> (K, V)
PyObject* kv_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded<8>(n, [&]() -> PyObject* {
    const Call c(a[0]);
    const Pool p(c, a[0], a[1], a[2], a[3]);
    if (!THPDtype_Check(a[5])) throw Decline{};
    const at::ScalarType type = reinterpret_cast<THPDtype*>(a[5])->scalar_type;
    if (code_of(type) == kBad) throw Decline{};
    const at::Tensor& s = c.on(a[4]);
    if (s.dim() != 1) throw Decline{};
    const int64_t T = s.size(0);
    void* slots = c.dense(a[4], at::kLong, {T});
    at::Tensor kv[2];
    int64_t ld[2];
    for (int i = 0; i < 2; ++i) {
      kv[i] = a[6 + i] == Py_None ? c.make({T, p.heads, p.dim}, type) : c.on(a[6 + i]);
      if (kv[i].scalar_type() != type) throw Decline{};
      ld[i] = c.heads(kv[i], T, p.heads, p.dim);
    }
    call([&] {
      return gptq_kv_read(p.data, p.pages, p.page, p.heads, p.dim, (const int64_t*)slots, T, kv[0].data_ptr(), kv[1].data_ptr(),
                          code_of(type), ld[0], ld[1], c.stream);
    });
    PyObject *k = back(a[6], kv[0]), *v = back(a[7], kv[1]);
    PyObject* both = k && v ? PyTuple_Pack(2, k, v) : nullptr;
    Py_XDECREF(k);
    Py_XDECREF(v);
    return both;
  });
}

// pool, page_size, n_kv_heads, head_dim, Q, cu_q, kv_lens, block_table, max_q, sm_scale, causal, window, O, lse, ws -> O
PyObject* kv_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded<15>(n, [&]() -> PyObject* {
    const Call c(a[4]);
    const Pool p(c, a[0], a[1], a[2], a[3]);
    const at::Tensor &Q = c.on(a[4]), &table = c.on(a[7]);
    const at::ScalarType type = Q.scalar_type();
    if (type != at::kBFloat16 && type != at::kHalf) throw Decline{};
    const int64_t ldq = c.heads(Q, -1, -1, p.dim), total = Q.size(0), hq = Q.size(1);
    if (table.scalar_type() != at::kInt || table.dim() != 2) throw Decline{};
    const int64_t batch = table.size(0), width = table.size(1);
    if (batch < 1 || width < 1 || table.stride(1) != 1) throw Decline{};
    void* cu = c.dense(a[5], at::kInt, {batch + 1});
    void* lens = c.dense(a[6], at::kInt, {batch});
    const int64_t max_q = integer(a[8]), window = integer(a[11]);
    const float scale = a[9] == Py_None ? (float)(1.0 / std::sqrt((double)p.dim)) : real(a[9]);
    const at::Tensor O = a[12] == Py_None ? c.make({total, hq, p.dim}, type) : c.on(a[12]);
    if (O.scalar_type() != type) throw Decline{};
    const int64_t ldo = c.heads(O, total, hq, p.dim);
    void* lse = c.dense_or_null(a[13], at::kFloat, {total, hq});
    at::Tensor own;
    size_t bytes = 0;
    void* ws = c.workspace(a[14], gptq_kv_attention_workspace_size(total, (int)hq, p.heads, p.dim, batch, max_q), bytes, own);
    const bool causal = flag(a[10]);
    call([&] {
      return gptq_kv_attention(Q.data_ptr(), code_of(type), total, (int)hq, p.heads, p.dim, ldq, (const int32_t*)cu,
                               (const int32_t*)lens, (const int32_t*)table.data_ptr(), batch > 1 ? table.stride(0) : width,
                               width, batch, max_q, p.data, p.pages, p.page, scale, causal, window, O.data_ptr(), ldo,
                               (float*)lse, ws, bytes, c.stream);
    });
    return back(a[12], O);
  });
}

template <typename F>
PyCFunction fast(F f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)); }

PyMethodDef methods[] = {{"adapter_linear", fast(adapter_linear), METH_FASTCALL, nullptr},
                         {"qk_norm_rope", fast(qk_norm_rope), METH_FASTCALL, nullptr},
                         {"add_rms_norm", fast(add_rms_norm), METH_FASTCALL, nullptr},
                         {"linear", fast(linear), METH_FASTCALL, nullptr},
                         {"sample", fast(sample), METH_FASTCALL, nullptr},
                         {"kv_append", fast(kv_append), METH_FASTCALL, nullptr},
                         {"kv_read", fast(kv_read), METH_FASTCALL, nullptr},
                         {"kv_attention", fast(kv_attention), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "serving_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_serving_calls() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "built_for", BUILT_FOR) != 0) Py_CLEAR(m);
  return m;
}
