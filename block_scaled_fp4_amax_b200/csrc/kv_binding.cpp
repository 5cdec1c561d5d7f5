// kv_binding.cpp — Python binding of the key/value cache's entry points (fp4_kv_append, fp4_kv_read,
// fp4_kv_attention of include/fp4mx.h): checks of the tensors and argument marshalling, nothing else.
//
// The other entry points go through ctypes.  These three are called once a layer and token, with
// fifteen tensors and sizes among them, and in Python their checks alone took longer than the kernels
// of a small decoding step (attention over 300 tokens: 28 us a call on the host, 8 on the GPU).
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <optional>
#include <sstream>

#include "../../include/fp4mx.h"

namespace {

using at::Tensor;

std::string describe(const Tensor& t) {
  std::ostringstream s;
  s << t.scalar_type() << " " << t.sizes() << " (strides " << t.strides() << ") on " << t.device();
  return s.str();
}

const Tensor& tensor(PyObject* o, const char* name) {
  TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a torch.Tensor, not ", Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}

long long integer(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    TORCH_CHECK_TYPE(false, name, " must be an integer of 64 bits, not ", Py_TYPE(o)->tp_name);
  }
  return v;
}

int integer32(PyObject* o, const char* name) {
  const long long v = integer(o, name);
  TORCH_CHECK_VALUE(v >= INT_MIN && v <= INT_MAX, name, " is out of range: ", v);
  return (int)v;
}

bool on(const Tensor& t, int dev) { return t.is_cuda() && t.get_device() == dev; }

// The cache's arrays and the format with its scales.
struct Cache {
  unsigned char *kq, *ks, *vq, *vs;
  long pages;
  int page, heads, dim, block, dev;
  fp4_format fmt;
  const float *kg = nullptr, *vg = nullptr;
};

Cache cache_of(PyObject* const* a, PyObject* fmt, PyObject* k_global, PyObject* v_global) {
  const Tensor &kq = tensor(a[0], "kq"), &ks = tensor(a[1], "ks"), &vq = tensor(a[2], "vq"), &vs = tensor(a[3], "vs");
  TORCH_CHECK_VALUE(kq.is_cuda() && kq.dim() == 4, "kq: expected a CUDA tensor [pages, heads, page, head_dim / 2], got ", describe(kq));
  Cache c;
  c.fmt = (fp4_format)integer32(fmt, "fmt");
  c.dev = kq.get_device();
  c.block = c.fmt == FP4_MXFP4 ? 32 : 16;
  const int64_t pages = kq.size(0), heads = kq.size(1), page = kq.size(2), half = kq.size(3);
  TORCH_CHECK_VALUE(heads <= INT_MAX && page <= INT_MAX && half <= INT_MAX / 2, "kq: extents out of range: ", describe(kq));
  const int64_t rows[4] = {pages, heads, page, half}, blocks[4] = {pages, heads, page, 2 * half / c.block};
  const Tensor* all[4] = {&kq, &ks, &vq, &vs};
  for (int i = 0; i < 4; ++i) {
    const Tensor& t = *all[i];
    const at::IntArrayRef want(i % 2 ? blocks : rows, 4);
    TORCH_CHECK_VALUE(t.scalar_type() == at::kByte && t.sizes() == want && t.is_contiguous() && on(t, c.dev),
                      "cache array ", i, ": expected a contiguous uint8 tensor ", want, " on cuda:", c.dev, ", got ", describe(t));
  }
  c.kq = kq.data_ptr<uint8_t>();
  c.ks = ks.data_ptr<uint8_t>();
  c.vq = vq.data_ptr<uint8_t>();
  c.vs = vs.data_ptr<uint8_t>();
  c.pages = pages;
  c.page = (int)page;
  c.heads = (int)heads;
  c.dim = (int)(2 * half);
  PyObject* g[2] = {k_global, v_global};
  for (int i = 0; i < 2; ++i) {
    if (g[i] == Py_None) continue;
    const Tensor& t = tensor(g[i], "k_global, v_global");
    TORCH_CHECK_VALUE(t.scalar_type() == at::kFloat && t.numel() == 1 && on(t, c.dev),
                      "k_global, v_global: expected float32 tensors of one element on cuda:", c.dev, ", got ", describe(t));
    (i ? c.vg : c.kg) = t.data_ptr<float>();
  }
  return c;
}

// A contiguous vector of integers (int32 or int64) of n elements (n < 0: any number).
const Tensor& integers(PyObject* o, const char* name, at::ScalarType type, int64_t n, int dev) {
  const Tensor& t = tensor(o, name);
  TORCH_CHECK_VALUE(t.scalar_type() == type && t.dim() == 1 && (n < 0 || t.size(0) == n) && t.is_contiguous() && on(t, dev), name,
                    ": expected a contiguous ", type, " vector of ", n < 0 ? std::string("any number of") : std::to_string(n),
                    " elements on cuda:", dev, ", got ", describe(t));
  return t;
}

struct Table {
  const int* p;
  long stride;
  int cols, seqs;
};
Table table_of(PyObject* o, int64_t seqs, int dev) {
  const Tensor& t = tensor(o, "block table");
  TORCH_CHECK_VALUE(t.scalar_type() == at::kInt && t.dim() == 2 && t.size(0) == seqs && on(t, dev) && (t.size(1) <= 1 || t.stride(1) == 1) &&
                        t.size(1) <= INT_MAX && seqs <= INT_MAX,
                    "block table: expected an int32 tensor [", seqs, ", pages] with adjacent entries on cuda:", dev, ", got ", describe(t));
  return {t.data_ptr<int>(), (long)(seqs > 1 ? t.stride(0) : t.size(1)), (int)t.size(1), (int)seqs};
}

// Token and head strides of a [tokens, heads, head_dim] tensor with adjacent channels (an extent of one
// has none that matters).
struct Strides {
  long token, head;
};
Strides strided(const Tensor& t, const char* name, int64_t tokens, int64_t heads, int64_t dim, int dev) {
  TORCH_CHECK_VALUE(t.dim() == 3 && t.size(0) == tokens && t.size(1) == heads && t.size(2) == dim && on(t, dev) &&
                        (t.numel() == 0 || t.stride(2) == 1),
                    name, ": expected [", tokens, ", ", heads, ", ", dim, "] with adjacent channels on cuda:", dev, ", got ", describe(t));
  return {(long)(tokens > 1 ? t.stride(0) : 0), (long)(heads > 1 ? t.stride(1) : 0)};
}

fp4_dtype dtype_of(const Tensor& t) {
  if (t.scalar_type() == at::kBFloat16) return FP4_BF16;
  TORCH_CHECK_TYPE(t.scalar_type() == at::kFloat, "input dtype must be float32 or bfloat16, got ", t.scalar_type());
  return FP4_F32;
}

// The call's stream made current, with its device: torch's current one on `dev` (stream None), or the
// caller's (a tuple of its id, device and device type).  Tensors allocated meanwhile belong to it.
struct On {
  std::optional<c10::cuda::CUDAGuard> device;
  std::optional<c10::cuda::CUDAStreamGuard> guard;
  void* stream;
  On(PyObject* s, int dev) {
    if (s == Py_None) {
      if (c10::cuda::current_device() != dev) device.emplace((c10::DeviceIndex)dev);
      stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
      return;
    }
    TORCH_CHECK_TYPE(PyTuple_Check(s) && PyTuple_GET_SIZE(s) == 3, "stream: expected a torch.cuda.Stream");
    const auto st = c10::cuda::CUDAStream::unpack3(integer(PyTuple_GET_ITEM(s, 0), "stream id"),
                                                   (c10::DeviceIndex)integer32(PyTuple_GET_ITEM(s, 1), "stream device"),
                                                   (c10::DeviceType)integer32(PyTuple_GET_ITEM(s, 2), "stream device type"));
    TORCH_CHECK_VALUE(st.device_index() == dev, "the stream belongs to cuda:", (int)st.device_index(), ", the cache to cuda:", dev);
    guard.emplace(st);
    stream = st.stream();
  }
};

#define KV_ARGS(n) TORCH_CHECK_TYPE(nargs == (n), "expected ", (n), " arguments, got ", nargs)

// (k, v, kq, ks, vq, vs, slots, fmt, mode, k_global, v_global, stream) -> status
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  KV_ARGS(12);
  const Cache c = cache_of(a + 2, a[7], a[9], a[10]);
  const Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
  const int64_t tokens = k.dim() == 3 ? k.size(0) : 0;
  const Strides ks = strided(k, "k", tokens, c.heads, c.dim, c.dev), vs = strided(v, "v", tokens, c.heads, c.dim, c.dev);
  TORCH_CHECK_VALUE(v.scalar_type() == k.scalar_type(), "k and v differ in dtype: ", k.scalar_type(), " and ", v.scalar_type());
  const fp4_dtype dt = dtype_of(k);
  const Tensor& slots = integers(a[6], "slots", at::kLong, tokens, c.dev);
  const On s(a[11], c.dev);
  return PyLong_FromLong(fp4_kv_append(k.data_ptr(), v.data_ptr(), dt, (long)tokens, ks.token, ks.head, vs.token, vs.head,
                                       reinterpret_cast<const long long*>(slots.data_ptr<int64_t>()), c.fmt, c.block,
                                       integer32(a[8], "mode"), c.kg, c.vg, c.kq, c.ks, c.vq, c.vs, c.pages, c.page, c.heads, c.dim,
                                       s.stream));
  END_HANDLE_TH_ERRORS
}

// (kq, ks, vq, vs, table, cu, total, fmt, starts, out is bf16, k_global, v_global, k_out, v_out, stream)
//   -> (k, v) or status
PyObject* kv_read(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  KV_ARGS(15);
  const Cache c = cache_of(a, a[7], a[10], a[11]);
  const Tensor& cu = integers(a[5], "cu", at::kInt, -1, c.dev);
  TORCH_CHECK_VALUE(cu.size(0) >= 1, "cu: expected seqs + 1 elements, got none");
  const int64_t seqs = cu.size(0) - 1;
  const int* starts = a[8] == Py_None ? nullptr : integers(a[8], "starts", at::kInt, seqs, c.dev).data_ptr<int>();
  const Table t = table_of(a[4], seqs, c.dev);
  const long long total = integer(a[6], "total");
  TORCH_CHECK_VALUE(total >= 0, "total is negative: ", total);
  const On s(a[14], c.dev);
  Tensor k, v;
  const int64_t shape[3] = {total, c.heads, c.dim};
  if (a[12] == Py_None) {
    const auto opt = at::TensorOptions().device(at::kCUDA, (c10::DeviceIndex)c.dev).dtype(a[9] == Py_True ? at::kBFloat16 : at::kFloat);
    k = at::empty(at::IntArrayRef(shape, 3), opt);
    v = at::empty(at::IntArrayRef(shape, 3), opt);
  } else {
    k = tensor(a[12], "out");
    v = tensor(a[13], "out");
    for (const Tensor* o : {&k, &v})
      TORCH_CHECK_VALUE(o->sizes() == at::IntArrayRef(shape, 3) && o->scalar_type() == k.scalar_type() && o->is_contiguous() && on(*o, c.dev),
                        "out: expected two contiguous tensors ", at::IntArrayRef(shape, 3), " of one dtype on cuda:", c.dev, ", got ", describe(*o));
  }
  const fp4_status st = fp4_kv_read(c.kq, c.ks, c.vq, c.vs, c.pages, c.page, c.heads, c.dim, c.fmt, c.block, c.kg, c.vg, t.p, t.stride,
                                    t.cols, t.seqs, cu.data_ptr<int>(), starts, (long)total, dtype_of(k), k.data_ptr(), v.data_ptr(), s.stream);
  if (st != FP4_OK) return PyLong_FromLong(st);
  return PyTuple_Pack(2, THPObjectPtr(THPVariable_Wrap(k)).get(), THPObjectPtr(THPVariable_Wrap(v)).get());
  END_HANDLE_TH_ERRORS
}

// (q, kq, ks, vq, vs, table, lens, fmt, cu_q, max_q, scale, causal, window, want_lse, k_global, v_global, out,
//  workspace, stream) -> (out, lse or None) or status
PyObject* kv_attention(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  KV_ARGS(19);
  const Cache c = cache_of(a + 1, a[7], a[14], a[15]);
  const Tensor& q = tensor(a[0], "q");
  TORCH_CHECK_VALUE(q.dim() == 3 && q.size(1) <= INT_MAX, "q: expected [tokens, query heads, ", c.dim, "], got ", describe(q));
  const int64_t total = q.size(0), heads = q.size(1);
  const Strides qs = strided(q, "q", total, heads, c.dim, c.dev);
  const fp4_dtype dt = dtype_of(q);
  const Tensor& lens = integers(a[6], "lens", at::kInt, -1, c.dev);
  const int64_t seqs = lens.size(0);
  const int* cu = a[8] == Py_None ? nullptr : integers(a[8], "cu_q", at::kInt, seqs + 1, c.dev).data_ptr<int>();
  const Table t = table_of(a[5], seqs, c.dev);
  const int max_q = integer32(a[9], "max_q"), window = integer32(a[12], "window");
  const double scale = PyFloat_AsDouble(a[10]);
  if (scale == -1.0 && PyErr_Occurred()) return nullptr;
  const int causal = PyObject_IsTrue(a[11]), want_lse = PyObject_IsTrue(a[13]);
  if (causal < 0 || want_lse < 0) return nullptr;
  const On s(a[18], c.dev);
  const auto opt = at::TensorOptions().device(at::kCUDA, (c10::DeviceIndex)c.dev);
  Tensor out, lse, ws;
  if (a[16] == Py_None) {
    out = at::empty(q.sizes(), opt.dtype(at::kBFloat16));
  } else {
    out = tensor(a[16], "out");
    TORCH_CHECK_VALUE(out.sizes() == q.sizes() && out.scalar_type() == at::kBFloat16 && out.is_contiguous() && on(out, c.dev),
                      "out: expected a contiguous bfloat16 tensor ", q.sizes(), " on cuda:", c.dev, ", got ", describe(out));
  }
  if (want_lse) lse = at::empty({total, heads}, opt.dtype(at::kFloat));
  if (a[17] == Py_None) {
    ws = at::empty({(int64_t)fp4_workspace_size(FP4_OP_KV_ATTENTION, (long)total, (long)heads)}, opt.dtype(at::kByte));
  } else {
    ws = tensor(a[17], "workspace");
    TORCH_CHECK_VALUE(ws.is_contiguous() && on(ws, c.dev), "workspace: expected a contiguous tensor on cuda:", c.dev, ", got ", describe(ws));
  }
  const fp4_status st = fp4_kv_attention(
      q.data_ptr(), dt, (long)total, qs.token, qs.head, (int)heads, c.kq, c.ks, c.vq, c.vs, c.pages, c.page, c.heads, c.dim, c.fmt, c.block,
      c.kg, c.vg, t.p, t.stride, t.cols, t.seqs, cu, max_q, lens.data_ptr<int>(), (float)scale, causal, window, out.data_ptr(),
      want_lse ? lse.data_ptr<float>() : nullptr, ws.data_ptr(), ws.nbytes(), s.stream);
  if (st != FP4_OK) return PyLong_FromLong(st);
  THPObjectPtr o(THPVariable_Wrap(out)), l;
  if (want_lse) {
    l = THPVariable_Wrap(lse);
  } else {
    Py_INCREF(Py_None);
    l = Py_None;
  }
  return PyTuple_Pack(2, o.get(), l.get());
  END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"kv_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(kv_append)), METH_FASTCALL, nullptr},
    {"kv_read", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(kv_read)), METH_FASTCALL, nullptr},
    {"kv_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(kv_attention)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kv_binding", "Checks and marshalling of the key/value cache's calls.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kv_binding() { return PyModule_Create(&module); }
