// Calls of the operators on block-scaled caches from Python, for the case that every
// argument is as the operator wants it: the checks of api.py on tensors, and the library's
// entry point on torch's current stream.  A function returns the entry point's status, or
// None where an argument is not plainly right (and nothing was enqueued): api.py's own
// checks then say what is wrong, allocate what is missing, or change the device.  Ten to
// thirty attribute reads and as many converted arguments cost a call 7 to 16 us from
// Python; here they cost less than one.
#include <Python.h>

#include <algorithm>
#include <cstdint>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "kattn.h"

namespace {

// The library's entry points, set once: the library is not linked to this module.
decltype(&kattn_rope) entry_rope = nullptr;
decltype(&kattn_append_blocks) entry_append = nullptr;
decltype(&kattn_read_blocks) entry_read = nullptr;
decltype(&kattn_decode_blocks) entry_decode = nullptr;

struct NotPlain {};                        // an argument that api.py has to look at

const at::Tensor& tensor(PyObject* o) {
  if (!THPVariable_Check(o)) throw NotPlain();
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda() || t.layout() != at::kStrided) throw NotPlain();
  return t;
}
long long integer(PyObject* o) {
  if (!PyLong_Check(o)) throw NotPlain();
  int over = 0;
  const long long v = PyLong_AsLongLongAndOverflow(o, &over);
  if (over || v > INT32_MAX || v < INT32_MIN) throw NotPlain();
  return v;
}
int truth(PyObject* o) {
  if (o == Py_True) return 1;
  if (o == Py_False) return 0;
  throw NotPlain();
}
void want(bool b) {
  if (!b) throw NotPlain();
}
int type_code(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return KATTN_F32;
    case at::kBFloat16: return KATTN_BF16;
    case at::kHalf: return KATTN_F16;
    default: throw NotPlain();
  }
}

// Tensors of one call: all on the current device.
struct Call {
  int device = -1;
  void on(const at::Tensor& t) {
    if (device < 0) {
      device = t.get_device();
      want(device == c10::cuda::current_device());
    }
    want(t.get_device() == device);
  }
  const at::Tensor& plain(PyObject* o, at::ScalarType type, int dims) {
    const at::Tensor& t = tensor(o);
    on(t);
    want(t.scalar_type() == type && t.dim() == dims && t.is_contiguous());
    return t;
  }
  // [rows][heads][128], rows at a stride of their own
  const at::Tensor& heads(PyObject* o, int64_t* stride) {
    const at::Tensor& t = tensor(o);
    on(t);
    want(t.dim() == 3 && t.size(2) == KATTN_HEAD_DIM && t.size(0) <= INT32_MAX && t.size(1) <= INT32_MAX);
    if (t.numel()) want(t.stride(2) == 1 && (t.size(1) == 1 || t.stride(1) == KATTN_HEAD_DIM));
    *stride = t.size(0) > 1 ? t.stride(0) : std::max<int64_t>(t.size(1), 1) * KATTN_HEAD_DIM;
    return t;
  }
  void* stream() const { return c10::cuda::getCurrentCUDAStream(device).stream(); }
};

struct Cache {
  void *k, *v;
  float *k_scale, *v_scale;
  int code, Hkv, cap, block_rows;
  Cache(Call& c, PyObject* const* a) {             // k, k_scale, v, v_scale
    const at::Tensor& tk = tensor(a[0]);
    code = tk.scalar_type() == at::kChar ? KATTN_INT8 : KATTN_E4M3;
    const at::ScalarType type = code == KATTN_INT8 ? at::kChar : at::kFloat8_e4m3fn;
    c.plain(a[0], type, 3);
    const at::Tensor& tv = c.plain(a[2], type, 3);
    const at::Tensor& ks = c.plain(a[1], at::kFloat, 2);
    const at::Tensor& vs = c.plain(a[3], at::kFloat, 2);
    const int64_t blocks = ks.size(1);
    want(tk.sizes() == tv.sizes() && tk.size(2) == KATTN_HEAD_DIM && ks.size(0) == tk.size(0) &&
         vs.sizes() == ks.sizes() && blocks >= 1 && tk.size(1) % blocks == 0 && tk.size(0) <= INT32_MAX &&
         tk.size(1) <= INT32_MAX);
    k = tk.data_ptr();
    v = tv.data_ptr();
    k_scale = static_cast<float*>(ks.data_ptr());
    v_scale = static_cast<float*>(vs.data_ptr());
    Hkv = (int)tk.size(0);
    cap = (int)tk.size(1);
    block_rows = (int)(tk.size(1) / blocks);
  }
};

const int32_t* list(Call& c, PyObject* o, int64_t n) {
  const at::Tensor& t = c.plain(o, at::kInt, 1);
  want(t.size(0) == n);
  return static_cast<const int32_t*>(t.data_ptr());
}
const at::Tensor& block_table(Call& c, PyObject* o) {
  const at::Tensor& t = c.plain(o, at::kInt, 2);
  want(t.size(0) <= INT32_MAX && t.size(1) <= INT32_MAX);
  return t;
}
const at::Tensor& angles(Call& c, PyObject* o) {
  const at::Tensor& t = c.plain(o, at::kFloat, 3);
  want(t.size(2) == 2 && t.size(0) <= INT32_MAX && t.size(1) <= KATTN_HEAD_DIM);
  return t;
}

template <typename F>
PyObject* run(Py_ssize_t n, Py_ssize_t wanted, F&& body) {
  try {
    if (n != wanted) throw NotPlain();
    return PyLong_FromLong(body());
  } catch (...) {                                  // (torch's own errors too: api.py meets them again)
    PyErr_Clear();
    Py_RETURN_NONE;
  }
}
// The library's work without Python's lock, as a launch may wait for room in the queue.
template <typename F>
int unlocked(F&& f) {
  struct Unlock {
    PyThreadState* s = PyEval_SaveThread();
    ~Unlock() { PyEval_RestoreThread(s); }
  } unlock;
  return f();
}

// x, positions, table, interleaved, out
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return run(n, 5, [&]() -> int {
    Call c;
    int64_t xs, os;
    const at::Tensor& x = c.heads(a[0], &xs);
    const at::Tensor& out = c.heads(a[4], &os);
    const int xt = type_code(x.scalar_type()), ot = type_code(out.scalar_type());
    want(out.sizes() == x.sizes() && (ot == xt || ot == KATTN_F32));
    const int32_t* positions = list(c, a[1], x.size(0));
    const at::Tensor& table = angles(c, a[2]);
    const int inter = truth(a[3]);
    if (x.size(0) == 1 && x.data_ptr() == out.data_ptr()) os = xs;
    return unlocked([&] {
      return entry_rope(x.data_ptr(), xt, (int)x.size(0), (int)x.size(1), KATTN_HEAD_DIM, xs, positions,
                        static_cast<const float*>(table.data_ptr()), (int)table.size(0), 2 * (int)table.size(1),
                        inter, out.data_ptr(), ot, os, c.stream());
    });
  });
}

// k_new, v_new, cu_rows, start, k, k_scale, v, v_scale, block_table, page_rows, table,
// interleaved, q, q_out, workspace
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return run(n, 15, [&]() -> int {
    Call c;
    int64_t ks, vs, qs = 0, qos = 0;
    const at::Tensor& kn = c.heads(a[0], &ks);
    const at::Tensor& vn = c.heads(a[1], &vs);
    const at::ScalarType type = kn.scalar_type();
    const int xt = type_code(type);
    const Cache cache(c, a + 4);
    want(vn.scalar_type() == type && vn.sizes() == kn.sizes() && kn.size(1) == cache.Hkv);
    const at::Tensor& table = block_table(c, a[8]);
    const int64_t B = table.size(0);
    const int32_t* cu = list(c, a[2], B + 1);
    const int32_t* start = list(c, a[3], B);
    const int page = (int)integer(a[9]), inter = truth(a[11]);
    const float* turns = nullptr;
    int positions = 0, rot = 0, Hq = 0;
    if (a[10] != Py_None) {
      const at::Tensor& t = angles(c, a[10]);
      turns = static_cast<const float*>(t.data_ptr());
      positions = (int)t.size(0);
      rot = 2 * (int)t.size(1);
    }
    const void* q = nullptr;
    void* q_out = nullptr;
    want((a[12] == Py_None) == (a[13] == Py_None));
    if (a[12] != Py_None) {
      const at::Tensor& tq = c.heads(a[12], &qs);
      const at::Tensor& to = c.heads(a[13], &qos);
      want(turns && tq.scalar_type() == type && to.scalar_type() == type && tq.size(0) == kn.size(0) &&
           to.sizes() == tq.sizes());
      q = tq.data_ptr();
      q_out = to.data_ptr();
      Hq = (int)tq.size(1);
      if (tq.size(0) == 1 && q == q_out) qos = qs;
    }
    const at::Tensor& ws = c.plain(a[14], at::kByte, 1);
    return unlocked([&] {
      return entry_append(kn.data_ptr(), vn.data_ptr(), xt, (int)kn.size(0), cache.Hkv, KATTN_HEAD_DIM, ks, vs, cu,
                          start, (int)B, cache.k, cache.k_scale, cache.v, cache.v_scale, cache.code, cache.cap,
                          cache.block_rows, static_cast<const int32_t*>(table.data_ptr()), (int)table.size(1), page,
                          turns, positions, rot, inter, q, Hq, qs, q_out, qos, ws.data_ptr(), (size_t)ws.numel(),
                          c.stream());
    });
  });
}

// k, k_scale, v, v_scale, block_table, page_rows, cu_rows, start, n_rows, out_k, out_v, workspace
PyObject* read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return run(n, 12, [&]() -> int {
    Call c;
    const Cache cache(c, a);
    const at::Tensor& table = block_table(c, a[4]);
    const int64_t B = table.size(0), rows = integer(a[8]);
    const int32_t* cu = list(c, a[6], B + 1);
    const int32_t* start = list(c, a[7], B);
    const at::Tensor& tk = tensor(a[9]);
    const at::ScalarType type = tk.scalar_type();
    const int ot = type_code(type);
    c.plain(a[9], type, 3);
    const at::Tensor& tv = c.plain(a[10], type, 3);
    want(tk.size(0) == rows && tk.size(1) == cache.Hkv && tk.size(2) == KATTN_HEAD_DIM && tv.sizes() == tk.sizes());
    const int page = (int)integer(a[5]);
    const at::Tensor& ws = c.plain(a[11], at::kByte, 1);
    return unlocked([&] {
      return entry_read(cache.k, cache.k_scale, cache.v, cache.v_scale, cache.code, cache.Hkv, KATTN_HEAD_DIM,
                        cache.cap, cache.block_rows, static_cast<const int32_t*>(table.data_ptr()),
                        (int)table.size(1), page, cu, start, (int)B, (int)rows, tk.data_ptr(), tv.data_ptr(), ot,
                        ws.data_ptr(), (size_t)ws.numel(), c.stream());
    });
  });
}

// q, k, k_scale, v, v_scale, block_table, page_rows, ctx_len, max_ctx, out, sm_scale, workspace
PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return run(n, 12, [&]() -> int {
    Call c;
    const at::Tensor& tq = tensor(a[0]);
    const at::ScalarType type = tq.scalar_type();
    const int qt = type_code(type);
    c.plain(a[0], type, 4);
    const Cache cache(c, a + 1);
    const at::Tensor& out = c.plain(a[9], type, 4);
    const at::Tensor& table = block_table(c, a[5]);
    const int64_t B = tq.size(0);
    want(tq.size(3) == KATTN_HEAD_DIM && out.sizes() == tq.sizes() && table.size(0) == B && cache.Hkv >= 1 &&
         tq.size(1) <= INT32_MAX && tq.size(2) <= INT32_MAX && tq.size(2) % cache.Hkv == 0);
    const int32_t* ctx = list(c, a[7], B);
    const int page = (int)integer(a[6]), max_ctx = (int)integer(a[8]);
    want(max_ctx > 0 && max_ctx < 1 << 30 && PyFloat_Check(a[10]));
    const float scale = (float)PyFloat_AS_DOUBLE(a[10]);
    const at::Tensor& ws = c.plain(a[11], at::kByte, 1);
    return unlocked([&] {
      return entry_decode(tq.data_ptr(), qt, cache.k, cache.k_scale, cache.v, cache.v_scale, cache.code, cache.cap,
                          cache.block_rows, static_cast<const int32_t*>(table.data_ptr()), (int)table.size(1), page,
                          ctx, (int)B, (int)tq.size(1), (int)tq.size(2), cache.Hkv, KATTN_HEAD_DIM, max_ctx, scale,
                          out.data_ptr(), ws.data_ptr(), (size_t)ws.numel(), c.stream());
    });
  });
}

// The addresses of the entry points, in the order above.
PyObject* setup(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void* at[4];
  for (Py_ssize_t i = 0; i < 4; ++i) {
    at[i] = n == 4 ? PyLong_AsVoidPtr(a[i]) : nullptr;
    if (!at[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "four addresses of entry points");
      return nullptr;
    }
  }
  entry_rope = reinterpret_cast<decltype(entry_rope)>(at[0]);
  entry_append = reinterpret_cast<decltype(entry_append)>(at[1]);
  entry_read = reinterpret_cast<decltype(entry_read)>(at[2]);
  entry_decode = reinterpret_cast<decltype(entry_decode)>(at[3]);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"setup", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(setup)), METH_FASTCALL, nullptr},
    {"rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(rope)), METH_FASTCALL, nullptr},
    {"append_blocks", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(append)), METH_FASTCALL, nullptr},
    {"read_blocks", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(read)), METH_FASTCALL, nullptr},
    {"decode_blocks", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(decode)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_bind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// torch_version: the torch that this was compiled against; api.py uses it with no other.
PyMODINIT_FUNC PyInit__bind() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "torch_version", KATTN_TORCH_VERSION) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
