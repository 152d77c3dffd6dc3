// The Python side of the calls that a decode step issues every few
// microseconds (wq_kv_write, wq_kv_read, wq_attn_decode, wq_rope): asks the
// tensors for types, shapes and strides, allocates outputs, and calls the C
// ABI with the current stream.  In the interpreter the same questions and the
// marshalling cost more than the kernels (a decode step's rotary positions:
// 9 us there, 4.6 here, of which the launch is 2.3).
//
// Every function returns its result, or the library's status (a negative
// int), which the caller turns into an exception with the library's message.
// The library's functions are handed over by address, so that this module
// uses the one that the package has loaded.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <ATen/ops/empty.h>
#include <c10/hip/HIPStream.h>

#include <cmath>
#include <cstdint>
#include <memory>

#include "../../include/wq.h"

namespace {

decltype(&wq_kv_write) kv_write_fn;
decltype(&wq_kv_read) kv_read_fn;
decltype(&wq_attn_decode_workspace) workspace_fn;
decltype(&wq_attn_decode) attn_fn;
decltype(&wq_rope) rope_fn;

void *stream() { return c10::hip::getCurrentHIPStream().stream(); }

const at::Tensor &tensor(PyObject *o, const char *name) {
  TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor, got ", Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}

struct Rows {
  int64_t rows, cols, ld;
  uint16_t *data;
};

// fp16 GPU rows [rows][cols] of any row stride
Rows rows(const at::Tensor &t, const char *name) {
  TORCH_CHECK_VALUE(t.is_cuda() && t.scalar_type() == at::kHalf, name, " must be a float16 GPU tensor");
  TORCH_CHECK_VALUE(t.dim() == 2, name, " must be [rows][columns], got ", t.sizes());
  Rows r{t.size(0), t.size(1), 0, static_cast<uint16_t *>(t.data_ptr())};
  TORCH_CHECK_VALUE(r.cols <= 1 || t.stride(1) == 1, name, " must have contiguous rows, got strides ", t.strides());
  r.ld = r.rows > 1 ? t.stride(0) : r.cols;   // a single row's stride is arbitrary
  return r;
}

const int32_t *ints(const at::Tensor &t, const char *name) {
  TORCH_CHECK_VALUE(t.is_cuda() && t.scalar_type() == at::kInt && t.is_contiguous(), name,
                    " must be a contiguous int32 GPU tensor");
  return static_cast<const int32_t *>(t.data_ptr());
}

at::Tensor make(int64_t r, int64_t c, const at::Tensor &like) {
  return at::empty({r, c}, at::TensorOptions().dtype(at::kHalf).device(like.device()));
}

int64_t integer(PyObject *o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}

void expect_args(Py_ssize_t n, Py_ssize_t want) { TORCH_CHECK_TYPE(n == want, want, " arguments expected, ", n, " given"); }

// A cache as Python holds it: the descriptor, and the tensors it describes.
struct Cache {
  static constexpr int kTensors = 5;
  wq_kv_cache c;
  at::Tensor t[kTensors];       // k, v, k_params, v_params, signs; some undefined
  size_t bytes[kTensors];
};
constexpr char kCacheName[] = "wq_kv_cache";
const char *const kTensorNames[Cache::kTensors] = {"k", "v", "k_params", "v_params", "signs"};

void free_cache(PyObject *o) { delete static_cast<Cache *>(PyCapsule_GetPointer(o, kCacheName)); }

// The descriptor with the addresses that the tensors have at this call (a
// tensor's storage can be replaced under it).  An integer is the address of
// a descriptor that the caller keeps up itself.
const wq_kv_cache *cache_at(PyObject *o) {
  if (!PyCapsule_CheckExact(o)) {
    const wq_kv_cache *c = reinterpret_cast<const wq_kv_cache *>(integer(o));
    TORCH_CHECK_VALUE(c && c->head_dim > 0, "no cache");
    return c;
  }
  Cache *h = static_cast<Cache *>(PyCapsule_GetPointer(o, kCacheName));
  if (!h) throw python_error();
  void *at[Cache::kTensors];
  for (int i = 0; i < Cache::kTensors; ++i) {
    const at::Tensor &t = h->t[i];
    at[i] = t.defined() ? t.data_ptr() : nullptr;
    TORCH_CHECK_VALUE(!t.defined() || (t.nbytes() == h->bytes[i] && t.is_contiguous() && t.is_cuda()), kTensorNames[i],
                      " is not the contiguous GPU tensor of ", h->bytes[i],
                      " bytes that was described: assign resized tensors to the KVCache");
  }
  h->c.k = at[0];
  h->c.v = at[1];
  h->c.k_params = static_cast<uint16_t *>(at[2]);
  h->c.v_params = static_cast<uint16_t *>(at[3]);
  h->c.rht_signs = static_cast<const uint32_t *>(at[4]);
  return &h->c;
}

// cache(address, k, v, k_params, v_params, signs): a descriptor's copy and its tensors (or None), for the calls below
PyObject *cache(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect_args(n, 1 + Cache::kTensors);
  auto h = std::make_unique<Cache>();
  h->c = *cache_at(a[0]);
  for (int i = 0; i < Cache::kTensors; ++i) {
    if (a[1 + i] == Py_None) continue;
    h->t[i] = tensor(a[1 + i], kTensorNames[i]);
    h->bytes[i] = h->t[i].nbytes();
  }
  PyObject *o = PyCapsule_New(h.get(), kCacheName, free_cache);
  if (!o) throw python_error();
  h.release();
  return o;
  END_HANDLE_TH_ERRORS
}

// bind(kv_write, kv_read, workspace, attn, rope): the library's functions
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect_args(n, 5);
  kv_write_fn = reinterpret_cast<decltype(kv_write_fn)>(integer(a[0]));
  kv_read_fn = reinterpret_cast<decltype(kv_read_fn)>(integer(a[1]));
  workspace_fn = reinterpret_cast<decltype(workspace_fn)>(integer(a[2]));
  attn_fn = reinterpret_cast<decltype(attn_fn)>(integer(a[3]));
  rope_fn = reinterpret_cast<decltype(rope_fn)>(integer(a[4]));
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// kv_write(cache, k, v, slots)
PyObject *kv_write(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect_args(n, 4);
  const wq_kv_cache *c = cache_at(a[0]);
  const at::Tensor &tk = tensor(a[1], "k"), &tv = tensor(a[2], "v"), &ts = tensor(a[3], "slots");
  const Rows k = rows(tk, "k"), v = rows(tv, "v");
  const int32_t *slots = ints(ts, "slots");
  const int64_t tokens = ts.numel(), cols = (int64_t)c->kv_heads * c->head_dim;
  TORCH_CHECK_VALUE(k.cols == cols && v.cols == cols && k.rows == tokens && v.rows == tokens, "k ", tk.sizes(), " and v ",
                    tv.sizes(), " are not [", tokens, " slots][", cols, " channels]");
  return PyLong_FromLong(kv_write_fn(c, k.data, k.ld, v.data, v.ld, slots, tokens, stream()));
  END_HANDLE_TH_ERRORS
}

// kv_read(cache, slots, out): out None or a pair
PyObject *kv_read(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect_args(n, 3);
  const wq_kv_cache *c = cache_at(a[0]);
  const at::Tensor &ts = tensor(a[1], "slots");
  const int32_t *slots = ints(ts, "slots");
  const int64_t tokens = ts.numel(), cols = (int64_t)c->kv_heads * c->head_dim;
  at::Tensor tk, tv;
  if (a[2] == Py_None) {
    tk = make(tokens, cols, ts);
    tv = make(tokens, cols, ts);
  } else {
    THPObjectPtr two(PySequence_Tuple(a[2]));
    if (!two) throw python_error();
    TORCH_CHECK_VALUE(PyTuple_GET_SIZE(two.get()) == 2, "out must be a pair of tensors");
    tk = tensor(PyTuple_GET_ITEM(two.get(), 0), "out[0]");
    tv = tensor(PyTuple_GET_ITEM(two.get(), 1), "out[1]");
  }
  const Rows k = rows(tk, "out[0]"), v = rows(tv, "out[1]");
  TORCH_CHECK_VALUE(k.cols == cols && v.cols == cols && k.rows == tokens && v.rows == tokens, "out ", tk.sizes(), " and ",
                    tv.sizes(), " are not [", tokens, " slots][", cols, " channels]");
  const wq_status st = kv_read_fn(c, slots, tokens, k.data, k.ld, v.data, v.ld, stream());
  if (st != WQ_OK) return PyLong_FromLong(st);
  THPObjectPtr pk(THPVariable_Wrap(std::move(tk))), pv(THPVariable_Wrap(std::move(tv)));
  if (!pk || !pv) throw python_error();
  return PyTuple_Pack(2, pk.get(), pv.get());
  END_HANDLE_TH_ERRORS
}

// attn_decode(cache, q, table, lens, max_len, window, scale, workspace, out); max_len, scale,
// workspace and out may be None
PyObject *attn_decode(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect_args(n, 9);
  const wq_kv_cache *c = cache_at(a[0]);
  const at::Tensor &tq = tensor(a[1], "q"), &tt = tensor(a[2], "table"), &tl = tensor(a[3], "lens");
  const Rows q = rows(tq, "q");
  const int64_t heads = q.cols / c->head_dim;
  TORCH_CHECK_VALUE(heads * c->head_dim == q.cols && heads <= INT32_MAX, "q: ", q.cols, " columns are not heads of ",
                    c->head_dim);
  TORCH_CHECK_VALUE(tt.is_cuda() && tt.scalar_type() == at::kInt, "table must be an int32 GPU tensor");
  TORCH_CHECK_VALUE(tt.dim() == 2 && tt.size(0) == q.rows, "table must be [", q.rows, "][pages], got ", tt.sizes());
  const int64_t pages = tt.size(1), held = pages * c->page_size;
  TORCH_CHECK_VALUE(pages <= 1 || tt.stride(1) == 1, "table must have contiguous rows, got strides ", tt.strides());
  const int32_t *lens = ints(tl, "lens");
  TORCH_CHECK_VALUE(tl.dim() == 1 && tl.size(0) == q.rows, "lens must be [", q.rows, "], got ", tl.sizes());
  const int64_t max_len = a[4] == Py_None ? held : integer(a[4]), window = integer(a[5]);
  TORCH_CHECK_VALUE(max_len <= held, "max_len=", max_len, ": ", pages, " pages of ", c->page_size, " tokens hold ", held);
  double scale = 1.0 / std::sqrt((double)c->head_dim);
  if (a[6] != Py_None) {
    scale = PyFloat_AsDouble(a[6]);
    if (scale == -1.0 && PyErr_Occurred()) throw python_error();
  }
  at::Tensor ty = a[8] == Py_None ? make(q.rows, q.cols, tq) : tensor(a[8], "out");
  const Rows y = rows(ty, "out");
  TORCH_CHECK_VALUE(y.rows == q.rows && y.cols == q.cols, "out must be [", q.rows, "][", q.cols, "], got ", ty.sizes());
  at::Tensor tw;
  size_t bytes = 0;
  if (a[7] == Py_None) {
    bytes = workspace_fn(c, q.rows, (int32_t)heads, max_len, window);
    if (bytes == (size_t)-1) return PyLong_FromLong(WQ_E_ARG);
    if (bytes) tw = at::empty({(int64_t)bytes}, at::TensorOptions().dtype(at::kByte).device(tq.device()));
  } else {
    tw = tensor(a[7], "workspace");
    TORCH_CHECK_VALUE(tw.is_cuda() && tw.is_contiguous(), "workspace must be a contiguous GPU tensor");
    bytes = tw.nbytes();
  }
  const wq_status st =
      attn_fn(c, q.data, q.ld, (int32_t)heads, q.rows, static_cast<const int32_t *>(tt.data_ptr()),
              q.rows > 1 ? tt.stride(0) : pages, lens, max_len, window, (float)scale, y.data, y.ld,
              tw.defined() ? tw.data_ptr() : nullptr, bytes, stream());
  return st != WQ_OK ? PyLong_FromLong(st) : THPVariable_Wrap(std::move(ty));
  END_HANDLE_TH_ERRORS
}

// rope(xs, cos, sin, positions, head_dim, pair_axis, adjacent, out); pair_axis bytes or None, out None or a sequence
PyObject *rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect_args(n, 8);
  THPObjectPtr xs(PySequence_Tuple(a[0])), outs(a[7] == Py_None ? PyTuple_New(0) : PySequence_Tuple(a[7]));
  if (!xs || !outs) throw python_error();
  const Py_ssize_t count = PyTuple_GET_SIZE(xs.get());
  TORCH_CHECK_VALUE(count > 0 && count <= WQ_MAX_BATCH && (a[7] == Py_None || PyTuple_GET_SIZE(outs.get()) == count),
                    "xs: ", count, " arrays (1 to ", WQ_MAX_BATCH, "), and as many in out");
  const at::Tensor &tc = tensor(a[1], "cos"), &ts = tensor(a[2], "sin"), &tp = tensor(a[3], "positions");
  for (const at::Tensor *t : {&tc, &ts})
    TORCH_CHECK_VALUE(t->is_cuda() && t->scalar_type() == at::kFloat && t->is_contiguous(),
                      "cos and sin must be contiguous float32 GPU tensors");
  TORCH_CHECK_VALUE(tc.dim() == 2 && tc.sizes() == ts.sizes(), "cos and sin must be [rows][rot / 2], got ", tc.sizes(),
                    " and ", ts.sizes());
  const int32_t *positions = ints(tp, "positions");
  TORCH_CHECK_VALUE(tp.dim() == 1 || tp.dim() == 2, "positions must be [axes][tokens] or [tokens], got ", tp.sizes());
  const int64_t axes = tp.dim() == 2 ? tp.size(0) : 1, tokens = tp.size(-1), half = tc.size(1), head_dim = integer(a[4]);
  TORCH_CHECK_VALUE(head_dim > 0 && head_dim <= INT32_MAX && half <= INT32_MAX / 2 && axes <= INT32_MAX, "head_dim=", head_dim,
                    ", rot=", 2 * half, ", axes=", axes, " out of range");
  const uint8_t *axis = nullptr;
  if (a[5] != Py_None) {
    TORCH_CHECK_TYPE(PyBytes_Check(a[5]), "pair_axis must be bytes");
    TORCH_CHECK_VALUE(PyBytes_GET_SIZE(a[5]) == half, "pair_axis: ", PyBytes_GET_SIZE(a[5]), " entries for ", half, " pairs");
    axis = reinterpret_cast<const uint8_t *>(PyBytes_AS_STRING(a[5]));
  }
  const int adjacent = PyObject_IsTrue(a[6]);
  if (adjacent < 0) throw python_error();
  const uint16_t *px[WQ_MAX_BATCH];
  uint16_t *py[WQ_MAX_BATCH];
  int64_t ldx[WQ_MAX_BATCH], ldy[WQ_MAX_BATCH];
  int32_t heads[WQ_MAX_BATCH];
  at::Tensor ys[WQ_MAX_BATCH];
  for (Py_ssize_t i = 0; i < count; ++i) {
    const at::Tensor &t = tensor(PyTuple_GET_ITEM(xs.get(), i), "xs");
    const Rows x = rows(t, "xs");
    const int64_t h = x.cols / head_dim;
    TORCH_CHECK_VALUE(x.rows == tokens && h * head_dim == x.cols && h <= INT32_MAX, "an array of ", t.sizes(), " is not [",
                      tokens, "][heads * ", head_dim, "]");
    ys[i] = a[7] == Py_None ? make(x.rows, x.cols, t) : tensor(PyTuple_GET_ITEM(outs.get(), i), "out");
    const Rows y = rows(ys[i], "out");
    TORCH_CHECK_VALUE(y.rows == x.rows && y.cols == x.cols, "out must be [", x.rows, "][", x.cols, "], got ", ys[i].sizes());
    px[i] = x.data;
    ldx[i] = x.ld;
    py[i] = y.data;
    ldy[i] = y.ld;
    heads[i] = (int32_t)h;
  }
  const wq_status st =
      rope_fn((int32_t)count, px, ldx, py, ldy, heads, tokens, (int32_t)head_dim, (int32_t)(2 * half),
              static_cast<const float *>(tc.data_ptr()), static_cast<const float *>(ts.data_ptr()), tc.size(0), positions,
              tokens, (int32_t)axes, axis, adjacent ? WQ_ROPE_ADJACENT : 0u, stream());
  if (st != WQ_OK) return PyLong_FromLong(st);
  THPObjectPtr list(PyList_New(count));
  if (!list) throw python_error();
  for (Py_ssize_t i = 0; i < count; ++i) {
    PyObject *y = THPVariable_Wrap(std::move(ys[i]));
    if (!y) throw python_error();
    PyList_SET_ITEM(list.get(), i, y);
  }
  return list.release();
  END_HANDLE_TH_ERRORS
}

#define WQ_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {WQ_METHOD(bind), WQ_METHOD(cache), WQ_METHOD(kv_write), WQ_METHOD(kv_read), WQ_METHOD(attn_decode), WQ_METHOD(rope),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_wqpy", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__wqpy() { return PyModule_Create(&module); }
