// The binding's short way for calls whose host time counts: one look at all of a call's
// tensors in C++ (type, shape, contiguity, device, the current device) and the call itself
// on the current stream.  api.py's own checks take 6 us for nine tensors, these 0.3; what
// does not fit goes back to them (-1), and they say why.  No check is left out: a call is
// made here only where each of theirs would pass.
#include <torch/csrc/autograd/python_variable.h>
#include <torch/version.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <initializer_list>

#include "fdllm.h"

namespace {

using at::ScalarType;
using Sizes = std::initializer_list<int64_t>;

const at::Tensor* tensor(PyObject* o) {
  return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr;
}

// A call's tensors: ok stays true while they fit.
struct Call {
  int dev = -1;
  bool ok = true;

  // the first tensor of n dimensions: all others must be on its device, the current one
  const at::Tensor* first(PyObject* o, int n) {
    const at::Tensor* t = tensor(o);
    ok = t && t->is_cuda() && t->dim() == n && t->is_contiguous();
    if (ok) {
      dev = t->get_device();
      ok = dev == c10::cuda::current_device();
    }
    return t;
  }
  void* take(PyObject* o, ScalarType type, Sizes shape) {
    const at::Tensor* t = ok ? tensor(o) : nullptr;
    ok = t && t->is_cuda() && t->get_device() == dev && t->scalar_type() == type &&
         t->sizes() == at::IntArrayRef(shape) && t->is_contiguous();
    return ok ? t->data_ptr() : nullptr;
  }
  void* maybe(PyObject* o, ScalarType type, Sizes shape) {  // or None
    return o == Py_None ? nullptr : take(o, type, shape);
  }
  float* floats(PyObject* o, Sizes shape) {
    return static_cast<float*>(take(o, ScalarType::Float, shape));
  }
  int32_t* ints(PyObject* o, Sizes shape) {
    return static_cast<int32_t*>(take(o, ScalarType::Int, shape));
  }
  int32_t* maybe_ints(PyObject* o, Sizes shape) {
    return static_cast<int32_t*>(maybe(o, ScalarType::Int, shape));
  }
  void* workspace(PyObject* o, size_t* bytes) {
    const at::Tensor* t = ok ? tensor(o) : nullptr;
    ok = t && t->is_cuda() && t->get_device() == dev && t->scalar_type() == ScalarType::Byte &&
         t->is_contiguous();
    *bytes = ok ? (size_t)t->numel() : 0;
    return ok ? t->data_ptr() : nullptr;
  }
  // sizes that the C interface takes as int
  int dim(const at::Tensor* t, int i) {
    if (!ok) return 0;
    const int64_t n = t->size(i);
    if (n > INT32_MAX) ok = false;
    return (int)n;
  }
  void* stream() const { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }
};

int row_dtype(const at::Tensor* t) {
  if (t->scalar_type() == ScalarType::BFloat16) return FDLLM_BF16;
  return t->scalar_type() == ScalarType::Float ? FDLLM_F32 : -1;
}

// The interpreter's lock is given up around `call`, which must not throw.
template <typename F>
PyObject* run(const Call& c, F call) {
  if (!c.ok) return PyLong_FromLong(-1);
  int st;
  void* stream = c.stream();
  Py_BEGIN_ALLOW_THREADS
  st = call(stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

// An exception of torch's, or too few arguments: the caller's own checks say it better.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* guarded(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != N) return PyLong_FromLong(-1);
  try {
    return F(a);
  } catch (...) {
    return PyLong_FromLong(-1);
  }
}

// k_rows, v_rows, pos, k_cache, v_cache, k_scale, v_scale, workspace
template <bool WRITE>
PyObject* cache_rows(PyObject* const* a) {
  Call c;
  const at::Tensor* rows = c.first(a[0], 4);
  const at::Tensor* cache = c.ok ? tensor(a[3]) : nullptr;
  c.ok = cache && cache->dim() == 4;
  if (!c.ok) return PyLong_FromLong(-1);
  const int B = c.dim(rows, 0), R = c.dim(rows, 1), H = c.dim(rows, 2), dh = c.dim(rows, 3);
  const int N = c.dim(cache, 2), type = row_dtype(rows);
  c.ok = c.ok && type >= 0;
  void* kr = c.ok ? rows->data_ptr() : nullptr;
  void* vr = c.take(a[1], rows->scalar_type(), {B, R, H, dh});
  const int32_t* pos = c.ints(a[2], {B, R});
  void* kc = c.take(a[3], ScalarType::Float8_e4m3fn, {B, H, N, dh});
  void* vc = c.take(a[4], ScalarType::Float8_e4m3fn, {B, H, N, dh});
  float* ks = c.floats(a[5], {B, H, N});
  float* vs = c.floats(a[6], {B, H, N});
  size_t bytes;
  void* ws = c.workspace(a[7], &bytes);
  return run(c, [&](void* stream) {
    if (WRITE)
      return fdllm_cache_write_fp8(B, N, H, dh, R, type, kr, vr, pos, kc, vc, ks, vs, ws, bytes, stream);
    return fdllm_cache_read_fp8(B, N, H, dh, R, type, pos, kc, vc, ks, vs, kr, vr, ws, bytes, stream);
  });
}

// q, k_cache, v_cache, [k_scale, v_scale,] cache_len, parent, n_nodes, out, workspace
template <bool FP8>
PyObject* tree_attend(PyObject* const* a) {
  Call c;
  const at::Tensor* q = c.first(a[0], 4);
  const at::Tensor* cache = c.ok ? tensor(a[1]) : nullptr;
  c.ok = cache && cache->dim() == 4;
  if (!c.ok) return PyLong_FromLong(-1);
  const int B = c.dim(q, 0), T = c.dim(q, 1), Hq = c.dim(q, 2), dh = c.dim(q, 3);
  const int Hkv = c.dim(cache, 1), N = c.dim(cache, 2), type = row_dtype(q);
  c.ok = c.ok && type >= 0;
  const void* qp = c.ok ? q->data_ptr() : nullptr;
  const ScalarType kind = FP8 ? ScalarType::Float8_e4m3fn : q->scalar_type();
  void* kc = c.take(a[1], kind, {B, Hkv, N, dh});
  void* vc = c.take(a[2], kind, {B, Hkv, N, dh});
  const float* ks = FP8 ? c.floats(a[3], {B, Hkv, N}) : nullptr;
  const float* vs = FP8 ? c.floats(a[4], {B, Hkv, N}) : nullptr;
  a += FP8 ? 5 : 3;
  const int32_t* len = c.ints(a[0], {B});
  const int32_t* parent = c.maybe_ints(a[1], {B, T});
  const int32_t* nodes = c.maybe_ints(a[2], {B});
  void* out = c.take(a[3], q->scalar_type(), {B, T, (int64_t)Hq * dh});
  size_t bytes;
  void* ws = c.workspace(a[4], &bytes);
  return run(c, [&](void* stream) {
    if (FP8)
      return fdllm_tree_attend_fp8(B, N, Hq, Hkv, dh, T, type, qp, kc, vc, ks, vs, len, parent, nodes, out,
                                   ws, bytes, stream);
    return fdllm_tree_attend(B, N, Hq, Hkv, dh, T, type, qp, kc, vc, len, parent, nodes, out, ws, bytes,
                             stream);
  });
}

// target, draft, tok, n_draft, u, r, n_accept, next_tok, workspace
PyObject* chain_verify(PyObject* const* a) {
  Call c;
  const at::Tensor* draft = c.first(a[1], 3);
  if (!c.ok) return PyLong_FromLong(-1);
  const int B = c.dim(draft, 0), T = c.dim(draft, 1), V = c.dim(draft, 2);
  const float* target = c.floats(a[0], {B, (int64_t)T + 1, V});
  const float* dr = c.floats(a[1], {B, T, V});
  const int32_t* tok = c.ints(a[2], {B, T});
  const int32_t* n = c.maybe_ints(a[3], {B});
  const float* u = c.floats(a[4], {B, T});
  const float* r = c.floats(a[5], {B});
  int32_t* na = c.ints(a[6], {B});
  int32_t* nt = c.ints(a[7], {B});
  size_t bytes;
  void* ws = c.workspace(a[8], &bytes);
  return run(c, [&](void* stream) {
    return fdllm_chain_verify(B, T, V, target, dr, tok, n, u, r, na, nt, ws, bytes, stream);
  });
}

// target, tok, parent, n_nodes, u, r, path, n_accept, next_tok, workspace
PyObject* tree_verify(PyObject* const* a) {
  Call c;
  const at::Tensor* t = c.first(a[0], 3);
  if (!c.ok) return PyLong_FromLong(-1);
  const int B = c.dim(t, 0), T = c.dim(t, 1), V = c.dim(t, 2);
  const float* target = c.floats(a[0], {B, T, V});
  const int32_t* tok = c.ints(a[1], {B, T});
  const int32_t* parent = c.ints(a[2], {B, T});
  const int32_t* n = c.maybe_ints(a[3], {B});
  const float* u = c.floats(a[4], {B, T});
  const float* r = c.floats(a[5], {B});
  int32_t* path = c.ints(a[6], {B, T});
  int32_t* na = c.ints(a[7], {B});
  int32_t* nt = c.ints(a[8], {B});
  size_t bytes;
  void* ws = c.workspace(a[9], &bytes);
  return run(c, [&](void* stream) {
    return fdllm_tree_verify(B, T, V, target, tok, parent, n, u, r, path, na, nt, ws, bytes, stream);
  });
}

#define FDLLM_FAST(name, f, n) \
  {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<f, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    FDLLM_FAST("cache_write_fp8", cache_rows<true>, 8),
    FDLLM_FAST("cache_read_fp8", cache_rows<false>, 8),
    FDLLM_FAST("tree_attend", tree_attend<false>, 8),
    FDLLM_FAST("tree_attend_fp8", tree_attend<true>, 10),
    FDLLM_FAST("chain_verify", chain_verify, 9),
    FDLLM_FAST("tree_verify", tree_verify, 10),
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fast", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// torch_version: of the headers that this was compiled against, whose layouts it relies on
PyMODINIT_FUNC PyInit__fast() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "torch_version", TORCH_VERSION) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
