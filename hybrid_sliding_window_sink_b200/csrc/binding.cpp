// binding.cpp - the usual calls of the operators around a paged KV cache, marshalled in C++.
//
// A Python extension module (_call.so) between _lib.py and libmimo_attn.so. Each function takes
// the arguments of the public function of the same name, checks what _lib.py checks, allocates
// what is not given, and calls the C ABI on the current stream. Where anything is out of the
// ordinary (a check fails, another device than the current one, a status other than MIMO_OK,
// which launches nothing) it returns None and _lib.py goes through the call itself, with its
// errors. For one short call the Python checks, ctypes and three allocations took 21 us where the
// kernels take 7.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>

#include "mimo_attn.h"

namespace {

// The library's entry points, given by _lib.py when it has loaded the product library.
struct {
  decltype(&mimo_attn_prefill_first) prefill_first;
  decltype(&mimo_attn_decode_paged) decode_paged;
  decltype(&mimo_attn_decode_paged_fp8) decode_paged_fp8;
  decltype(&mimo_attn_decode_paged_workspace_size) workspace_size;
  decltype(&mimo_attn_cache_append_paged) append;
  decltype(&mimo_attn_cache_append_paged_fp8) append_fp8;
  decltype(&mimo_attn_verify_drafts) verify;
} fn = {};

PyObject* bind(PyObject*, PyObject* args) {
  unsigned long long a[7];
  if (!PyArg_ParseTuple(args, "KKKKKKK", &a[0], &a[1], &a[2], &a[3], &a[4], &a[5], &a[6])) return nullptr;
  fn.prefill_first = reinterpret_cast<decltype(fn.prefill_first)>(a[0]);
  fn.decode_paged = reinterpret_cast<decltype(fn.decode_paged)>(a[1]);
  fn.decode_paged_fp8 = reinterpret_cast<decltype(fn.decode_paged_fp8)>(a[2]);
  fn.workspace_size = reinterpret_cast<decltype(fn.workspace_size)>(a[3]);
  fn.append = reinterpret_cast<decltype(fn.append)>(a[4]);
  fn.append_fp8 = reinterpret_cast<decltype(fn.append_fp8)>(a[5]);
  fn.verify = reinterpret_cast<decltype(fn.verify)>(a[6]);
  Py_RETURN_NONE;
}

// Collects one call's arguments; ok turns false at the first that is not as usual.
struct Args {
  PyObject* const* a;
  int device = -1;            // the first tensor's, which has to be the current one
  bool ok = true;

  explicit Args(PyObject* const* args) : a(args) {
    if (THPVariable_Check(a[0]) && THPVariable_Unpack(a[0]).is_cuda()) device = THPVariable_Unpack(a[0]).get_device();
    ok = device >= 0 && device == c10::cuda::current_device();
  }

  // tensor i of that type on the device, contiguous unless it is a pool; sizes: -1 = any
  const at::Tensor* tensor(int i, at::ScalarType type, std::initializer_list<int64_t> sizes, bool dense = true) {
    static const at::Tensor none;
    if (!ok || !THPVariable_Check(a[i])) return fail(none);
    const at::Tensor& t = THPVariable_Unpack(a[i]);
    if (!t.is_cuda() || t.get_device() != device || t.scalar_type() != type || t.layout() != at::kStrided ||
        t.is_conj() || t.is_neg() || t.dim() != static_cast<int64_t>(sizes.size()) || (dense && !t.is_contiguous()))
      return fail(none);
    int d = 0;
    for (int64_t s : sizes) {
      const int64_t have = t.size(d++);
      if (have > INT_MAX || (s >= 0 && s != have)) return fail(none);
    }
    return &t;
  }
  const at::Tensor* fail(const at::Tensor& none) {
    ok = false;
    return &none;
  }
  bool given(int i) const { return a[i] != Py_None; }
  int integer(int i) {
    int overflow = 0;
    if (!ok || !PyLong_Check(a[i])) {
      ok = false;
      return 0;
    }
    const long v = PyLong_AsLongAndOverflow(a[i], &overflow);
    if (overflow || v > INT_MAX || v < INT_MIN) ok = false;
    return static_cast<int>(v);
  }
  float real(int i) {
    if (!ok || (!PyFloat_Check(a[i]) && !PyLong_Check(a[i]))) {
      ok = false;
      return 0.f;
    }
    const double v = PyFloat_AsDouble(a[i]);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      ok = false;
    }
    return static_cast<float>(v);
  }
  // True or False itself; _lib.py goes by the truth value of anything else
  bool flag(int i) {
    if (a[i] != Py_True && a[i] != Py_False) ok = false;
    return a[i] == Py_True;
  }
  static void* data(const at::Tensor* t) { return t ? t->data_ptr() : nullptr; }
};

// Pages of pools that are contiguous within a page, with the same distance between pages.
bool pool(const at::Tensor& t, long long& stride) {
  long long row = 1, size = 1;
  for (int64_t d = t.dim() - 1; d >= 1; --d) {
    if (t.size(d) < 1 || (t.size(d) > 1 && t.stride(d) != size)) return false;
    size *= t.size(d);
    if (d == 2) row = size;
  }
  if (t.size(0) < 1) return false;
  long long step = size / row;
  if (t.size(0) > 1) {
    if (t.stride(0) % row || t.stride(0) < size) return false;
    step = t.stride(0) / row;
  }
  if (stride >= 0 && step != stride) return false;
  stride = step;
  return true;
}

// A new tensor on t's device, without the dispatcher (and scratch straight from the allocator): one
// short paged decode 9.4 -> 8.4 us a call, a small verification 6.6 -> 6.2.
at::Tensor fresh(at::IntArrayRef sizes, at::ScalarType type, const at::Tensor& t) {
  return at::Tensor(at::detail::empty_cuda(sizes, type, t.device(), std::nullopt));
}

PyObject* pair(at::Tensor a, const at::Tensor* b) {
  PyObject* x = THPVariable_Wrap(std::move(a));
  PyObject* y = b ? THPVariable_Wrap(*b) : Py_NewRef(Py_None);
  if (!x || !y) {
    Py_XDECREF(x);
    Py_XDECREF(y);
    return nullptr;
  }
  PyObject* r = PyTuple_Pack(2, x, y);
  Py_DECREF(x);
  Py_DECREF(y);
  return r;
}

// Runs f; a C++ exception (no memory for an output, say) is one more call that is not usual: _lib.py
// makes it again and raises torch's own error.
template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const std::exception&) {
    if (PyErr_Occurred()) return nullptr;
    Py_RETURN_NONE;
  }
}

bool arity(Py_ssize_t have, Py_ssize_t want) {
  if (have != want) PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, have);
  return have == want;
}

// (q, k, v, k_scale, v_scale, block_table, lengths, sink, window, n_first, softmax_scale, want_lse)
PyObject* decode_paged(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (!arity(n, 12)) return nullptr;
  return guarded([&]() -> PyObject* {
    if (!fn.decode_paged) Py_RETURN_NONE;
    Args in{args};
    const bool fp8 = in.given(3);
    const auto type = fp8 ? at::kByte : at::kBFloat16;
    const at::Tensor* q = in.tensor(0, at::kBFloat16, {-1, -1, 192});
    const at::Tensor* k = in.tensor(1, type, {-1, -1, -1, 192}, false);
    if (!in.ok) Py_RETURN_NONE;
    const int64_t B = q->size(0), hq = q->size(1), N = k->size(0), page = k->size(1), hkv = k->size(2);
    const at::Tensor* v = in.tensor(2, type, {N, page, hkv, 128}, false);
    const at::Tensor *ks = nullptr, *vs = nullptr, *sink = nullptr;
    if (fp8) {
      ks = in.tensor(3, at::kFloat, {N, page, hkv}, false);
      vs = in.tensor(4, at::kFloat, {N, page, hkv}, false);
    }
    const at::Tensor* table = in.tensor(5, at::kInt, {B, -1});
    const at::Tensor* lengths = in.tensor(6, at::kInt, {B});
    if (in.given(7)) sink = in.tensor(7, at::kFloat, {hq});
    const int window = in.integer(8), first = in.integer(9);
    const float scale = in.real(10);
    const bool want_lse = in.flag(11);
    long long stride = -1;
    if (!in.ok || !pool(*k, stride) || !pool(*v, stride) || (fp8 && (!pool(*ks, stride) || !pool(*vs, stride))))
      Py_RETURN_NONE;
    const mimo_shape shape{static_cast<int>(B), 1, static_cast<int>(hq), static_cast<int>(hkv), 192, 128, scale};
    const mimo_pages pages{static_cast<const int*>(table->data_ptr()), static_cast<int>(table->size(1)),
                           static_cast<int>(N), static_cast<int>(page), stride};
    const size_t bytes = fn.workspace_size(&shape, &pages, window, first);
    at::Tensor out = fresh({B, hq, 128}, at::kBFloat16, *q), lse;
    if (want_lse) lse = fresh({B, hq}, at::kFloat, *q);
    c10::DataPtr ws;                       // (goes back to the allocator in stream order)
    if (bytes) ws = c10::cuda::CUDACachingAllocator::get()->allocate(bytes);
    void* st = c10::cuda::getCurrentCUDAStream().stream();
    float* l = lse.defined() ? static_cast<float*>(lse.data_ptr()) : nullptr;
    void* w = ws.get();
    const int* len = static_cast<const int*>(lengths->data_ptr());
    const float* sk = static_cast<const float*>(Args::data(sink));
    const mimo_status rc =
        fp8 ? fn.decode_paged_fp8(&shape, q->data_ptr(), k->data_ptr(), v->data_ptr(), static_cast<float*>(ks->data_ptr()),
                                  static_cast<float*>(vs->data_ptr()), &pages, len, window, first, sk, out.data_ptr(), l,
                                  w, bytes, st)
            : fn.decode_paged(&shape, q->data_ptr(), k->data_ptr(), v->data_ptr(), &pages, len, window, first, sk,
                              out.data_ptr(), l, w, bytes, st);
    if (rc != MIMO_OK) Py_RETURN_NONE;
    return pair(std::move(out), lse.defined() ? &lse : nullptr);
  });
}

// (k_new, v_new, k, v, k_scale, v_scale, block_table, positions, n_new, rope_theta, rot_dims): True
PyObject* append_paged(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (!arity(n, 11)) return nullptr;
  return guarded([&]() -> PyObject* {
    if (!fn.append) Py_RETURN_NONE;
    Args in{args};
    const bool fp8 = in.given(4);
    const auto type = fp8 ? at::kByte : at::kBFloat16;
    const at::Tensor* kn = in.tensor(0, at::kBFloat16, {-1, -1, -1, 192});
    if (!in.ok) Py_RETURN_NONE;
    const int64_t B = kn->size(0), len = kn->size(1), hkv = kn->size(2);
    const at::Tensor* vn = in.tensor(1, at::kBFloat16, {B, len, hkv, 128});
    const at::Tensor* k = in.tensor(2, type, {-1, -1, hkv, 192}, false);
    if (!in.ok) Py_RETURN_NONE;
    const int64_t N = k->size(0), page = k->size(1);
    const at::Tensor* v = in.tensor(3, type, {N, page, hkv, 128}, false);
    const at::Tensor *ks = nullptr, *vs = nullptr, *count = nullptr;
    if (fp8) {
      ks = in.tensor(4, at::kFloat, {N, page, hkv}, false);
      vs = in.tensor(5, at::kFloat, {N, page, hkv}, false);
    }
    const at::Tensor* table = in.tensor(6, at::kInt, {B, -1});
    const at::Tensor* pos = in.tensor(7, at::kInt, {B});
    if (in.given(8)) count = in.tensor(8, at::kInt, {B});
    const float theta = in.real(9);
    const int rot = in.integer(10);
    long long stride = -1;
    if (!in.ok || !pool(*k, stride) || !pool(*v, stride) || (fp8 && (!pool(*ks, stride) || !pool(*vs, stride))))
      Py_RETURN_NONE;
    const mimo_shape shape{static_cast<int>(B), static_cast<int>(len), static_cast<int>(hkv), static_cast<int>(hkv), 192,
                           128, 0.f};
    const mimo_pages pages{static_cast<const int*>(table->data_ptr()), static_cast<int>(table->size(1)),
                           static_cast<int>(N), static_cast<int>(page), stride};
    void* st = c10::cuda::getCurrentCUDAStream().stream();
    const int* at0 = static_cast<const int*>(pos->data_ptr());
    const int* cnt = static_cast<const int*>(Args::data(count));
    const mimo_status rc =
        fp8 ? fn.append_fp8(&shape, kn->data_ptr(), vn->data_ptr(), at0, cnt, theta, rot, &pages, k->data_ptr(),
                            v->data_ptr(), static_cast<float*>(ks->data_ptr()), static_cast<float*>(vs->data_ptr()), st)
            : fn.append(&shape, kn->data_ptr(), vn->data_ptr(), at0, cnt, theta, rot, &pages, k->data_ptr(),
                        v->data_ptr(), st);
    if (rc != MIMO_OK) Py_RETURN_NONE;
    Py_RETURN_TRUE;
  });
}

// (q, k, v, sink, window, n_first, pos_offset, k_prefix_rotated, rope_theta, rot_dims, softmax_scale, want_lse)
PyObject* prefill_first(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (!arity(n, 12)) return nullptr;
  return guarded([&]() -> PyObject* {
    if (!fn.prefill_first) Py_RETURN_NONE;
    Args in{args};
    const at::Tensor* q = in.tensor(0, at::kBFloat16, {-1, -1, -1, 192});
    const int off = in.integer(6);
    const bool rotated = in.flag(7), want_lse = in.flag(11);
    if (!in.ok || off < 0) Py_RETURN_NONE;
    const int64_t B = q->size(0), len = q->size(1), hq = q->size(2);
    const at::Tensor* k = in.tensor(1, at::kBFloat16, {B, off + len, -1, 192});
    if (!in.ok) Py_RETURN_NONE;
    const int64_t hkv = k->size(2);
    const at::Tensor* v = in.tensor(2, at::kBFloat16, {B, off + len, hkv, 128});
    const at::Tensor* sink = in.given(3) ? in.tensor(3, at::kFloat, {hq}) : nullptr;
    const int window = in.integer(4), first = in.integer(5), rot = in.integer(9);
    const float theta = in.real(8), scale = in.real(10);
    if (!in.ok) Py_RETURN_NONE;
    const mimo_shape shape{static_cast<int>(B), static_cast<int>(len), static_cast<int>(hq), static_cast<int>(hkv), 192,
                           128, scale};
    at::Tensor out = fresh({B, len, hq, 128}, at::kBFloat16, *q), lse;
    if (want_lse) lse = fresh({B, hq, len}, at::kFloat, *q);
    const mimo_status rc = fn.prefill_first(
        &shape, q->data_ptr(), k->data_ptr(), v->data_ptr(), off, rotated, static_cast<float*>(Args::data(sink)),
        window, first, theta, rot, out.data_ptr(), lse.defined() ? static_cast<float*>(lse.data_ptr()) : nullptr,
        c10::cuda::getCurrentCUDAStream().stream());
    if (rc != MIMO_OK) Py_RETURN_NONE;
    return pair(std::move(out), lse.defined() ? &lse : nullptr);
  });
}

// (target_probs, draft_tokens, uniforms, draft_probs, n_valid)
PyObject* verify_drafts(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (!arity(n, 5)) return nullptr;
  return guarded([&]() -> PyObject* {
    if (!fn.verify) Py_RETURN_NONE;
    Args in{args};
    if (!in.ok) Py_RETURN_NONE;
    const at::ScalarType type = THPVariable_Unpack(args[0]).scalar_type();
    if (type != at::kFloat && type != at::kBFloat16) Py_RETURN_NONE;
    const at::Tensor* p = in.tensor(0, type, {-1, -1, -1});
    if (!in.ok || p->size(1) < 1) Py_RETURN_NONE;
    const int64_t B = p->size(0), T1 = p->size(1), V = p->size(2);
    const at::Tensor* draft = in.tensor(1, at::kInt, {B, T1 - 1});
    const at::Tensor* u = in.tensor(2, at::kFloat, {B, T1});
    const at::Tensor* q = in.given(3) ? in.tensor(3, type, {B, T1 - 1, V}) : nullptr;
    const at::Tensor* valid = in.given(4) ? in.tensor(4, at::kInt, {B}) : nullptr;
    if (!in.ok) Py_RETURN_NONE;
    at::Tensor acc = fresh({B}, at::kInt, *draft), tok = fresh({B, T1}, at::kInt, *draft);
    const mimo_status rc = fn.verify(
        static_cast<int>(B), static_cast<int>(T1 - 1), static_cast<int>(V),
        type == at::kFloat ? MIMO_PROBS_F32 : MIMO_PROBS_BF16, p->data_ptr(), Args::data(q),
        static_cast<int*>(draft->data_ptr()), static_cast<float*>(u->data_ptr()), static_cast<int*>(Args::data(valid)),
        static_cast<int*>(acc.data_ptr()), static_cast<int*>(tok.data_ptr()),
        c10::cuda::getCurrentCUDAStream().stream());
    if (rc != MIMO_OK) Py_RETURN_NONE;
    return pair(std::move(acc), &tok);
  });
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL
PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, "Addresses of the library's entry points."},
    {"decode_paged", FAST(decode_paged), "The usual call of _lib.decode_paged(_fp8), or None."},
    {"append_paged", FAST(append_paged), "The usual call of _lib.cache_append_paged(_fp8), or None."},
    {"prefill_first", FAST(prefill_first), "The usual call of _lib.prefill_first, or None."},
    {"verify_drafts", FAST(verify_drafts), "The usual call of _lib.verify_drafts, or None."},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_call", "Marshalling of the usual calls.", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__call() { return PyModule_Create(&module); }
