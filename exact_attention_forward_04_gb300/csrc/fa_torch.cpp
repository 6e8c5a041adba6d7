// The usual calls of the 4-bit cache and of rotary positions from PyTorch
// tensors to the C ABI: CUDA tensors of the current device, on its current
// stream.  A step of single tokens takes the GPU 3 to 10 us a call, and a call
// through Python's checks and ctypes takes the host 9 to 25; through here 4 to 10.
//
// Whatever is not usual (other types, shapes, positions [B, N], devices, a status other
// than FA_OK) gives None and nothing is enqueued: the Python function behind then makes
// the call itself and says what is wrong.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <cmath>

#include "fa_fwd.h"

namespace {

decltype(&fa_rope) g_rope;
decltype(&fa_cache_append_e2m1) g_append;
decltype(&fa_cache_read_e2m1) g_read;
decltype(&fa_cache_fwd_e2m1) g_forward;
decltype(&fa_cache_fwd_e2m1_workspace_size) g_workspace;

constexpr int64_t kInt = 0x7fffffff;

bool on_gpu(PyObject* o) { return THPVariable_Check(o) && THPVariable_Unpack(o).is_cuda(); }
// The tensor an argument is, if it is one of this type on the current device.
const at::Tensor* tensor(PyObject* o, at::ScalarType type, c10::DeviceIndex device) {
  if (!THPVariable_Check(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  return t.is_cuda() && t.scalar_type() == type && t.get_device() == device ? &t : nullptr;
}
const at::Tensor* vector(PyObject* o, at::ScalarType type, int64_t n, c10::DeviceIndex device) {
  const at::Tensor* t = tensor(o, type, device);
  return t && t->dim() == 1 && t->size(0) == n && t->is_contiguous() ? t : nullptr;
}
// bf16 [n, heads, d], a token's rows together, n > 0.
const at::Tensor* rows(PyObject* o, int64_t heads, int64_t d, c10::DeviceIndex device, int64_t& stride) {
  const at::Tensor* t = tensor(o, at::kBFloat16, device);
  if (!t || t->dim() != 3 || t->size(0) == 0 || t->size(0) > kInt || t->size(1) != heads || t->size(2) != d ||
      t->stride(2) != 1 || (heads > 1 && t->stride(1) != d))
    return nullptr;
  stride = t->size(0) > 1 ? t->stride(0) : heads * d;
  return t;
}
const at::Tensor* angles(PyObject* o, int64_t d, c10::DeviceIndex device) {
  const at::Tensor* t = tensor(o, at::kFloat, device);
  return t && t->dim() == 3 && t->size(2) == 2 && 2 * t->size(1) <= d && t->size(0) <= kInt && t->is_contiguous()
             ? t
             : nullptr;
}

struct Cache {
  const at::Tensor* data;
  int64_t blocks, H, P, d;
};
bool cache(PyObject* o, c10::DeviceIndex device, Cache& c) {
  c.data = tensor(o, at::kByte, device);
  if (!c.data || c.data->dim() != 4 || !c.data->is_contiguous() || c.data->size(3) % 18 != 0) return false;
  c.blocks = c.data->size(0);
  c.H = c.data->size(1);
  c.P = 16 * c.data->size(2);
  c.d = c.data->size(3) / 18;
  return c.H > 0 && c.d > 0 && c.blocks <= kInt && c.H <= kInt && c.P <= 128 && c.d <= 128;
}

at::Tensor make(c10::IntArrayRef sizes, at::ScalarType type, c10::DeviceIndex device) {
  return at::empty(sizes, at::TensorOptions().dtype(type).device(c10::Device(c10::kCUDA, device)));
}
void* stream(c10::DeviceIndex device) { return c10::cuda::getCurrentCUDAStream(device).stream(); }

bool flag(PyObject* o, int& f) {
  f = PyObject_IsTrue(o);
  if (f < 0) PyErr_Clear();
  return f >= 0;
}
bool number(PyObject* o, float& f) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  f = static_cast<float>(v);
  return true;
}

// `f` while other Python threads run: a launch waits while the GPU's queue is full, for
// as long as the work in front of it takes, and memory may have to be asked for.
template <typename F>
auto unlocked(F&& f) {
  struct Unlock {
    PyThreadState* state = PyEval_SaveThread();
    ~Unlock() { PyEval_RestoreThread(state); }
  } unlock;
  return f();
}

PyObject* pair(const at::Tensor& a, const at::Tensor& b) {
  PyObject* t = PyTuple_New(2);
  if (!t) return nullptr;
  PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(a));
  PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(b));
  return t;
}

// x, positions, table, interleaved, transposed
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 5 || !on_gpu(a[0])) Py_RETURN_NONE;
  const auto device = c10::cuda::current_device();
  const at::Tensor* x = tensor(a[0], at::kBFloat16, device);
  if (!x || (x->dim() != 3 && x->dim() != 4) || x->numel() == 0 || x->stride(x->dim() - 1) != 1) Py_RETURN_NONE;
  int interleaved, transposed;
  if (!flag(a[3], interleaved) || !flag(a[4], transposed)) Py_RETURN_NONE;
  const bool tokens = x->dim() == 3;
  const int64_t d = x->size(tokens ? 2 : 3), H = x->size(1), N = x->size(tokens ? 0 : 2), B = tokens ? 1 : x->size(0);
  const at::Tensor* pos = vector(a[1], at::kInt, N, device);
  const at::Tensor* table = angles(a[2], d, device);
  if (!pos || !table || d > 128 || B > kInt || H > kInt || N > kInt) Py_RETURN_NONE;
  at::Tensor out;
  const int st = unlocked([&] {
    out = make(x->sizes(), at::kBFloat16, device);
    const int64_t* xs = x->strides().data();
    return tokens ? g_rope(x->data_ptr(), 0, xs[1], xs[0], out.data_ptr(), 0, d, H * d,
                           static_cast<const int*>(pos->data_ptr()), 0, static_cast<const float*>(table->data_ptr()),
                           table->size(0), 1, H, N, d, 2 * table->size(1), interleaved, transposed, stream(device))
                  : g_rope(x->data_ptr(), xs[0], xs[1], xs[2], out.data_ptr(), H * N * d, N * d, d,
                           static_cast<const int*>(pos->data_ptr()), 0, static_cast<const float*>(table->data_ptr()),
                           table->size(0), B, H, N, d, 2 * table->size(1), interleaved, transposed, stream(device));
  });
  if (st != FA_OK) Py_RETURN_NONE;
  return THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

// k, v, data, k_unit, v_unit, slot_map, positions, table, interleaved: True where done
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 9 || !on_gpu(a[2])) Py_RETURN_NONE;
  const auto device = c10::cuda::current_device();
  Cache c;
  float ku, vu;
  int64_t ks, vs;
  int interleaved;
  if (!cache(a[2], device, c) || !number(a[3], ku) || !number(a[4], vu) || !flag(a[8], interleaved)) Py_RETURN_NONE;
  const at::Tensor* k = rows(a[0], c.H, c.d, device, ks);
  const at::Tensor* v = rows(a[1], c.H, c.d, device, vs);
  if (!k || !v || k->size(0) != v->size(0)) Py_RETURN_NONE;
  const int64_t T = k->size(0);
  const at::Tensor* slots = vector(a[5], at::kLong, T, device);
  const bool turned = a[6] != Py_None;
  if (!slots || turned != (a[7] != Py_None)) Py_RETURN_NONE;
  const at::Tensor* pos = turned ? vector(a[6], at::kInt, T, device) : nullptr;
  const at::Tensor* table = turned ? angles(a[7], c.d, device) : nullptr;
  if (turned && (!pos || !table)) Py_RETURN_NONE;
  const int st = unlocked([&] {
    return g_append(k->data_ptr(), v->data_ptr(), ks, vs, c.data->data_ptr(), ku, vu,
                    static_cast<const long long*>(slots->data_ptr()),
                    turned ? static_cast<const int*>(pos->data_ptr()) : nullptr,
                    turned ? static_cast<const float*>(table->data_ptr()) : nullptr, turned ? table->size(0) : 0,
                    turned ? 2 * table->size(1) : 0, interleaved, T, c.H, c.d, c.blocks, c.P, stream(device));
  });
  if (st != FA_OK) Py_RETURN_NONE;
  Py_RETURN_TRUE;
  END_HANDLE_TH_ERRORS
}

// data, k_unit, v_unit, slot_map: (k, v)
PyObject* read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 4 || !on_gpu(a[0])) Py_RETURN_NONE;
  const auto device = c10::cuda::current_device();
  Cache c;
  float ku, vu;
  if (!cache(a[0], device, c) || !number(a[1], ku) || !number(a[2], vu)) Py_RETURN_NONE;
  const at::Tensor* slots = tensor(a[3], at::kLong, device);
  if (!slots || slots->dim() != 1 || !slots->is_contiguous() || slots->size(0) == 0 || slots->size(0) > kInt)
    Py_RETURN_NONE;
  const int64_t T = slots->size(0);
  at::Tensor k, v;
  const int st = unlocked([&] {
    k = make({T, c.H, c.d}, at::kBFloat16, device);
    v = make({T, c.H, c.d}, at::kBFloat16, device);
    return g_read(c.data->data_ptr(), ku, vu, static_cast<const long long*>(slots->data_ptr()), k.data_ptr(),
                  v.data_ptr(), T, c.H, c.d, c.blocks, c.P, stream(device));
  });
  if (st != FA_OK) Py_RETURN_NONE;
  return pair(k, v);
  END_HANDLE_TH_ERRORS
}

// q, data, k_unit, v_unit, block_table, seq_lens, cu_q, scale, causal, workspace, slot_map: (o, lse)
PyObject* forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 11 || !on_gpu(a[1])) Py_RETURN_NONE;
  const auto device = c10::cuda::current_device();
  Cache c;
  float ku, vu, scale;
  int causal;
  if (!cache(a[1], device, c) || !number(a[2], ku) || !number(a[3], vu) || !flag(a[8], causal)) Py_RETURN_NONE;
  const at::Tensor* q = tensor(a[0], at::kBFloat16, device);
  if (!q || q->dim() != 3) Py_RETURN_NONE;
  const int64_t T = q->size(0), Hq = q->size(1);
  int64_t stride;
  if (Hq == 0 || Hq > kInt || Hq % c.H != 0 || !rows(a[0], Hq, c.d, device, stride)) Py_RETURN_NONE;
  const at::Tensor* table = tensor(a[4], at::kInt, device);
  if (!table || table->dim() != 2 || !table->is_contiguous() || table->size(0) == 0 || table->size(0) > kInt ||
      table->size(1) > kInt)
    Py_RETURN_NONE;
  const int64_t R = table->size(0), M = table->size(1);
  const at::Tensor* lens = vector(a[5], at::kInt, R, device);
  const at::Tensor* cu = vector(a[6], at::kInt, R + 1, device);
  const at::Tensor* slots = a[10] != Py_None ? vector(a[10], at::kLong, T, device) : nullptr;
  if (!lens || !cu || (a[10] != Py_None && !slots)) Py_RETURN_NONE;
  if (a[7] == Py_None) scale = static_cast<float>(1.0 / std::sqrt(static_cast<double>(c.d)));
  else if (!number(a[7], scale)) Py_RETURN_NONE;
  size_t bytes = 0;
  void* ws = nullptr;
  if (a[9] == Py_None) {
    bytes = g_workspace(R, T, Hq, c.H, c.d);
    if (bytes == 0) Py_RETURN_NONE;
  } else {
    if (!on_gpu(a[9])) Py_RETURN_NONE;
    const at::Tensor& given = THPVariable_Unpack(a[9]);
    if (given.get_device() != device || !given.is_contiguous()) Py_RETURN_NONE;
    bytes = given.nbytes();
    ws = given.data_ptr();
  }
  at::Tensor o, lse;
  const int st = unlocked([&] {
    at::Tensor mine;
    if (a[9] == Py_None) {
      mine = make({static_cast<int64_t>(bytes)}, at::kByte, device);
      ws = mine.data_ptr();
    }
    o = make({T, Hq, c.d}, at::kBFloat16, device);
    lse = make({T, Hq}, at::kFloat, device);
    return g_forward(q->data_ptr(), stride, c.data->data_ptr(), ku, vu, static_cast<const int*>(table->data_ptr()),
                     static_cast<const int*>(lens->data_ptr()), static_cast<const int*>(cu->data_ptr()),
                     slots ? static_cast<const long long*>(slots->data_ptr()) : nullptr, o.data_ptr(),
                     static_cast<float*>(lse.data_ptr()), R, T, Hq, c.H, c.d, c.blocks, c.P, M, scale, causal, ws,
                     bytes, stream(device));
  });
  if (st != FA_OK) Py_RETURN_NONE;
  return pair(o, lse);
  END_HANDLE_TH_ERRORS
}

// The addresses of fa_rope, fa_cache_append_e2m1, fa_cache_read_e2m1,
// fa_cache_fwd_e2m1 and fa_cache_fwd_e2m1_workspace_size in the loaded library.
PyObject* bind(PyObject*, PyObject* args) {
  unsigned long long p[5];
  if (!PyArg_ParseTuple(args, "KKKKK", p, p + 1, p + 2, p + 3, p + 4)) return nullptr;
  g_rope = reinterpret_cast<decltype(g_rope)>(p[0]);
  g_append = reinterpret_cast<decltype(g_append)>(p[1]);
  g_read = reinterpret_cast<decltype(g_read)>(p[2]);
  g_forward = reinterpret_cast<decltype(g_forward)>(p[3]);
  g_workspace = reinterpret_cast<decltype(g_workspace)>(p[4]);
  Py_RETURN_NONE;
}

template <typename F>
PyCFunction fast(F* f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f));
}
PyMethodDef methods[] = {{"bind", bind, METH_VARARGS, nullptr},
                         {"rope", fast(rope), METH_FASTCALL, nullptr},
                         {"append", fast(append), METH_FASTCALL, nullptr},
                         {"read", fast(read), METH_FASTCALL, nullptr},
                         {"forward", fast(forward), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "fa_torch", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit_fa_torch() { return PyModule_Create(&module_def); }
