// The Python binding of the calls whose kernels take a few microseconds: tensors are checked and
// turned into pointers here, in about a microsecond, where ctypes and Python's attribute lookups took
// ten. It holds no arithmetic; each function makes one call into libsvt.so, whose entry points it is
// given by address (bind), and returns the outputs, or the status of a refused call as an int.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <cuda_runtime_api.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cstring>
#include <initializer_list>

#include "svt.h"

namespace {

decltype(&svt_rope) g_rope = nullptr;
decltype(&svt_rope_append) g_rope_append = nullptr;
decltype(&svt_sparse_mla_backward_workspace_size) g_backward_ws = nullptr;
decltype(&svt_sparse_mla_backward) g_backward = nullptr;
decltype(&svt_distill_topk) g_distill = nullptr;

// What a function leaves through when a Python error has been set.
struct PyFailure {};

[[noreturn]] void type_error(const char* fmt, const char* name) {
  PyErr_Format(PyExc_TypeError, fmt, name);
  throw PyFailure{};
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) type_error("%s must be a tensor", name);
  return THPVariable_Unpack(o);
}
const at::Tensor* maybe(PyObject* o, const char* name) { return o == Py_None ? nullptr : &tensor(o, name); }

long long integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PyFailure{};
  return v;
}
int32_t int32(long long v) {
  if (v < INT_MIN || v > INT_MAX) {
    PyErr_SetString(PyExc_OverflowError, "a size or option does not fit 32 bits");
    throw PyFailure{};
  }
  return static_cast<int32_t>(v);
}
float real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PyFailure{};
  return static_cast<float>(v);
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw PyFailure{};
  return v != 0;
}

// The address of a contiguous tensor of this type and shape; null for null.
void* shaped(const at::Tensor* t, const char* name, at::ScalarType type, std::initializer_list<int64_t> shape) {
  if (t == nullptr) return nullptr;
  if (t->scalar_type() != type || t->dim() != static_cast<int64_t>(shape.size()) ||
      !std::equal(shape.begin(), shape.end(), t->sizes().begin()) || !t->is_contiguous())
    type_error("%s must be contiguous and of the type and shape the call documents", name);
  return t->data_ptr();
}

// The stream of a launch: `first` is on the current CUDA device (kernels are launched there, on its
// current stream) and every other given tensor beside it.
svt_stream_t launch_on(const at::Tensor& first, std::initializer_list<std::pair<const at::Tensor*, const char*>> others) {
  const c10::Device dev = first.device();
  if (!dev.is_cuda() || dev.index() != c10::cuda::current_device())
    type_error("%s must be on the current CUDA device", "tensors");
  for (const auto& o : others)
    if (o.first != nullptr && o.first->device() != dev) type_error("%s must be on the current CUDA device", o.second);
  return reinterpret_cast<svt_stream_t>(c10::cuda::getCurrentCUDAStream(dev.index()).stream());
}

// x [T, D] or [T, H, D] with unit column stride. A dimension of one row has no meaningful stride.
struct Rows {
  int64_t T, H, D, st, sh;
};
Rows rows_of(const at::Tensor& x, const char* name) {
  const auto n = x.sizes(), s = x.strides();
  if (n.size() != 2 && n.size() != 3) type_error("%s must be [T, D] or [T, H, D]", name);
  const bool three = n.size() == 3;
  Rows r;
  r.T = n[0];
  r.H = three ? n[1] : 1;
  r.D = n[three ? 2 : 1];
  r.st = r.T > 1 ? s[0] : r.H * r.D;
  r.sh = r.H > 1 ? s[1] : r.D;
  if (s[three ? 2 : 1] != 1 && r.D > 1) type_error("%s must have unit column stride", name);
  return r;
}

svt_kv_cache cache_of(const at::Tensor& data, PyObject* const* a) {
  svt_kv_cache kv;
  kv.data = data.data_ptr();
  kv.num_pages = integer(a[0]);
  kv.page_size = int32(integer(a[1]));
  kv.row_stride_bytes = int32(integer(a[2]));
  kv.dtype = static_cast<svt_kv_dtype>(integer(a[3]));
  if (!data.is_contiguous()) type_error("%s must be contiguous", "kv data");
  const int64_t row = kv.dtype == SVT_KV_BF16 ? 1152 : 656;
  const int64_t stride = kv.row_stride_bytes ? kv.row_stride_bytes : row;
  // descriptors out of range are left to the library's own checks
  if (kv.num_pages > 0 && kv.page_size > 0 && stride >= row && kv.num_pages < (1ll << 31) &&
      static_cast<int64_t>(data.nbytes()) < (kv.num_pages * kv.page_size - 1) * stride + row)
    type_error("%s holds fewer than num_pages * page_size rows", "kv data");
  return kv;
}

PyObject* wrap(at::Tensor t) { return THPVariable_Wrap(std::move(t)); }
PyObject* same(PyObject* o) {
  Py_INCREF(o);
  return o;
}

// rope(x, positions, freqs, offset, layout, inverse, amplitude, out or None)
PyObject* rope(PyObject* const* a) {
  const at::Tensor& x = tensor(a[0], "x");
  const auto type = x.scalar_type();
  if (type != at::kBFloat16 && type != at::kFloat) type_error("%s must be bf16 or fp32", "x");
  const Rows r = rows_of(x, "x");
  const at::Tensor &pos = tensor(a[1], "positions"), &freqs = tensor(a[2], "freqs");
  const at::Tensor* given = maybe(a[7], "out");
  if (given != nullptr && (given->scalar_type() != type || given->sizes() != x.sizes()))
    type_error("%s must have x's type and shape", "out");
  const svt_stream_t stream = launch_on(x, {{&pos, "positions"}, {&freqs, "freqs"}, {given, "out"}});
  const void* at = shaped(&pos, "positions", at::kInt, {r.T});
  const void* fr = shaped(&freqs, "freqs", at::kDouble, {freqs.numel()});
  at::Tensor made;
  if (given == nullptr) made = at::empty(x.sizes(), x.options());
  const at::Tensor& out = given ? *given : made;
  const Rows o = rows_of(out, "out");
  const svt_status st =
      g_rope(x.data_ptr(), out.data_ptr(), type == at::kFloat ? SVT_F32 : SVT_BF16, int32(r.T), int32(r.H), int32(r.D),
             r.st, r.sh, o.st, o.sh, static_cast<const int32_t*>(at), static_cast<const double*>(fr),
             int32(2 * freqs.numel()), int32(integer(a[3])), static_cast<svt_rope_layout>(integer(a[4])), real(a[6]),
             truth(a[5]), stream);
  if (st != SVT_OK) return PyLong_FromLong(st);
  return given ? same(a[7]) : wrap(made);
}

// rope_append(latent, k_rope, positions, slots, kv data, num_pages, page_size, row_stride, dtype, freqs, layout,
//             amplitude, q_rope or None, q_out or None, workspace)
PyObject* rope_append(PyObject* const* a) {
  const at::Tensor &lat = tensor(a[0], "latent"), &kr = tensor(a[1], "k_rope"), &pos = tensor(a[2], "positions"),
                   &slots = tensor(a[3], "slots"), &data = tensor(a[4], "kv data"), &freqs = tensor(a[9], "freqs"),
                   &ws = tensor(a[14], "workspace");
  const at::Tensor *q = maybe(a[12], "q_rope"), *qo = maybe(a[13], "q_out");
  const Rows l = rows_of(lat, "latent"), k = rows_of(kr, "k_rope");
  if (lat.scalar_type() != at::kBFloat16 || lat.dim() != 2 || l.D != 512)
    type_error("%s must be a bf16 [T, 512] tensor", "latent");
  if (kr.scalar_type() != at::kBFloat16 || kr.dim() != 2 || k.D != 64 || k.T != l.T)
    type_error("%s must be a bf16 [T, 64] tensor", "k_rope");
  if (q == nullptr && qo != nullptr) type_error("%s needs q_rope", "q_out");
  if (q != nullptr && (q->scalar_type() != at::kBFloat16 || q->dim() != 3 || q->size(0) != l.T || q->size(2) != 64))
    type_error("%s must be a bf16 [T, H, 64] tensor", "q_rope");
  if (qo != nullptr && (qo->scalar_type() != at::kBFloat16 || qo->sizes() != q->sizes()))
    type_error("%s must have q_rope's type and shape", "q_out");
  const svt_stream_t stream = launch_on(lat, {{&kr, "k_rope"}, {&pos, "positions"}, {&slots, "slots"}, {&data, "kv data"},
                                              {&freqs, "freqs"}, {&ws, "workspace"}, {q, "q_rope"}, {qo, "q_out"}});
  const svt_kv_cache kv = cache_of(data, a + 5);
  const void* at = shaped(&pos, "positions", at::kInt, {l.T});
  const void* sl = shaped(&slots, "slots", at::kInt, {l.T});
  const void* fr = shaped(&freqs, "freqs", at::kDouble, {32});
  at::Tensor made;
  if (q != nullptr && qo == nullptr) {
    made = at::empty(q->sizes(), q->options());
    qo = &made;
  }
  Rows qi{}, qd{};
  if (q != nullptr) {
    qi = rows_of(*q, "q_rope");
    qd = rows_of(*qo, "q_out");
  }
  const bool with_q = q != nullptr && qi.H > 0;
  const svt_status st = g_rope_append(
      lat.data_ptr(), l.st, kr.data_ptr(), k.st, static_cast<const int32_t*>(at), static_cast<const int32_t*>(sl),
      int32(l.T), &kv, static_cast<const double*>(fr), static_cast<svt_rope_layout>(integer(a[10])), real(a[11]),
      with_q ? q->data_ptr() : nullptr, int32(qi.H), qi.st, qi.sh, with_q ? qo->data_ptr() : nullptr, qd.st, qd.sh,
      ws.data_ptr(), ws.nbytes(), stream);
  if (st != SVT_OK) return PyLong_FromLong(st);
  return made.defined() ? wrap(made) : same(a[13]);
}

// sparse_mla_backward(q, kv data, num_pages, page_size, row_stride, dtype, topk, scale, out, lse, dout, dlse,
//                     block_table, seq_lens, req_of_token, topk_len, dq, dkv, return_weights, workspace).
// A workspace that is too small is answered by minus the bytes it needs.
PyObject* backward(PyObject* const* a) {
  const at::Tensor &q = tensor(a[0], "q"), &data = tensor(a[1], "kv data"), &topk = tensor(a[6], "topk"),
                   &out = tensor(a[8], "out"), &lse = tensor(a[9], "lse"), &dout = tensor(a[10], "dout"),
                   &ws = tensor(a[19], "workspace");
  const at::Tensor *dlse = maybe(a[11], "dlse"), *bt = maybe(a[12], "block_table"), *seq = maybe(a[13], "seq_lens"),
                   *req = maybe(a[14], "req_of_token"), *len = maybe(a[15], "topk_len"), *dq = maybe(a[16], "dq"),
                   *dkv = maybe(a[17], "dkv");
  if (q.scalar_type() != at::kBFloat16 || q.dim() != 3 || q.size(2) != 576 || !q.is_contiguous())
    type_error("%s must be a contiguous bf16 [T, H, 576] tensor", "q");
  const int64_t T = q.size(0), H = q.size(1);
  if (topk.dim() != 2 || topk.size(0) != T) type_error("%s must be an int32 [T, K] tensor", "topk");
  if (bt != nullptr && bt->dim() != 2) type_error("%s must be [num_reqs, max_blocks]", "block_table");
  const int64_t K = topk.size(1), reqs = bt ? bt->size(0) : 0, blocks = bt ? bt->size(1) : 0;
  const svt_stream_t stream =
      launch_on(q, {{&data, "kv data"}, {&topk, "topk"}, {&out, "out"}, {&lse, "lse"}, {&dout, "dout"}, {&ws, "workspace"},
                    {dlse, "dlse"}, {bt, "block_table"}, {seq, "seq_lens"}, {req, "req_of_token"}, {len, "topk_len"},
                    {dq, "dq"}, {dkv, "dkv"}});
  const svt_kv_cache kv = cache_of(data, a + 2);
  // (rows that no cache has are left to the library; a product that does not fit is none of dkv's)
  int64_t n = 0;
  if (__builtin_mul_overflow(kv.num_pages, static_cast<int64_t>(kv.page_size), &n)) n = -1;
  const auto i32 = at::kInt, f32 = at::kFloat, bf16 = at::kBFloat16;
  // an aligned address in the place of a tensor that has none; it is never read or written
  void* const any = reinterpret_cast<void*>(uintptr_t{256});
  const void* p_bt = shaped(bt, "block_table", i32, {reqs, blocks});
  if (bt != nullptr && bt->numel() == 0 && T > 0) p_bt = any;  // refused for its sizes: null would be no table
  const void* p_req = shaped(req, "req_of_token", i32, {T});
  const void* p_seq = bt ? shaped(seq, "seq_lens", i32, {reqs}) : nullptr;
  const void* p_topk = shaped(&topk, "topk", i32, {T, K});
  const void* p_len = shaped(len, "topk_len", i32, {T});
  const void* p_out = shaped(&out, "out", bf16, {T, H, 512});
  const void* p_lse = shaped(&lse, "lse", f32, {T, H});
  const void* p_dout = shaped(&dout, "dout", bf16, {T, H, 512});
  const void* p_dlse = shaped(dlse, "dlse", f32, {T, H});
  void* p_dq = shaped(dq, "dq", bf16, {T, H, 576});
  void* p_dkv = shaped(dkv, "dkv", bf16, {n, 576});
  const float scale = real(a[7]);
  auto call = [&](void* to_dq, void* to_dkv, float* to_weights, size_t ws_bytes) {
    return g_backward(q.data_ptr(), int32(T), int32(H), &kv, static_cast<const int32_t*>(p_bt), int32(reqs),
                      int32(blocks), static_cast<const int32_t*>(p_req), static_cast<const int32_t*>(p_seq),
                      static_cast<const int32_t*>(p_topk), int32(K), static_cast<const int32_t*>(p_len), scale, p_out,
                      static_cast<const float*>(p_lse), p_dout, static_cast<const float*>(p_dlse), to_dq, to_dkv,
                      to_weights, ws.data_ptr(), ws_bytes, stream);
  };
  svt_status st;
  const size_t need = g_backward_ws(int32(T), int32(H), int32(K), n);
  if (need <= 256 || n >= (1ll << 31) || ws.nbytes() < need) {  // (256: sizes that it takes for none)
    // A call without a workspace is refused, for that or for another reason, which comes first: only a call
    // that the library takes asks for its workspace, and the outputs are made within the sizes of one.
    st = call(dq ? p_dq : any, dkv ? p_dkv : any, nullptr, 0);
    return st != SVT_ERR_WORKSPACE ? PyLong_FromLong(st) : PyLong_FromLongLong(-static_cast<long long>(need));
  }
  at::Tensor made_q, made_kv, weights;
  if (dq == nullptr) {
    made_q = at::empty({T, H, 576}, q.options());
    p_dq = made_q.data_ptr();
  }
  if (dkv == nullptr) {
    made_kv = at::empty({n, 576}, q.options());
    p_dkv = made_kv.data_ptr();
  }
  if (truth(a[18])) weights = at::empty({T, K}, lse.options());
  st = call(p_dq, p_dkv, weights.defined() ? static_cast<float*>(weights.data_ptr()) : nullptr, ws.nbytes());
  if (st != SVT_OK) return PyLong_FromLong(st);
  PyObject* r = PyTuple_New(3);
  if (r == nullptr) return nullptr;
  PyTuple_SET_ITEM(r, 0, dq ? same(a[16]) : wrap(made_q));
  PyTuple_SET_ITEM(r, 1, dkv ? same(a[17]) : wrap(made_kv));
  PyTuple_SET_ITEM(r, 2, weights.defined() ? wrap(weights) : same(Py_None));
  return r;
}

// distill_topk(scores, topk, teacher, lens, temperature, kind, scope, row_weight, need_grad, dscores or None)
PyObject* distill(PyObject* const* a) {
  const at::Tensor &x = tensor(a[0], "scores"), &topk = tensor(a[1], "topk"), &teacher = tensor(a[2], "teacher");
  const at::Tensor *lens = maybe(a[3], "lens"), *rw = maybe(a[7], "row_weight"), *given = maybe(a[9], "dscores");
  const auto type = x.scalar_type();
  if ((type != at::kFloat && type != at::kBFloat16) || x.dim() != 2)
    type_error("%s must be an fp32 or bf16 [T, N] tensor", "scores");
  const Rows r = rows_of(x, "scores");
  const int64_t T = r.T, N = r.D;
  if (topk.dim() != 2 || topk.size(0) != T) type_error("%s must be an int32 [T, K] tensor", "topk");
  const int64_t K = topk.size(1);
  if (given != nullptr && (given->scalar_type() != type || given->sizes() != x.sizes()))
    type_error("%s must have scores' type and shape", "dscores");
  const svt_stream_t stream =
      launch_on(x, {{&topk, "topk"}, {&teacher, "teacher"}, {lens, "lens"}, {rw, "row_weight"}, {given, "dscores"}});
  const void* p_topk = shaped(&topk, "topk", at::kInt, {T, K});
  const void* p_teacher = shaped(&teacher, "teacher", at::kFloat, {T, K});
  const void* p_lens = shaped(lens, "lens", at::kInt, {T});
  const void* p_rw = shaped(rw, "row_weight", at::kFloat, {T});
  at::Tensor loss = at::empty({T}, x.options().dtype(at::kFloat)), made;
  const at::Tensor* grad = given;
  if (grad == nullptr && truth(a[8])) {
    made = at::empty({T, N}, x.options());
    grad = &made;
  }
  const Rows g = grad ? rows_of(*grad, "dscores") : r;
  const svt_status st = g_distill(
      x.data_ptr(), type == at::kFloat ? SVT_F32 : SVT_BF16, int32(T), int32(N), r.st, static_cast<const int32_t*>(p_lens),
      static_cast<const int32_t*>(p_topk), static_cast<const float*>(p_teacher), int32(K),
      static_cast<svt_teacher_kind>(integer(a[5])), static_cast<svt_distill_scope>(integer(a[6])), real(a[4]),
      static_cast<const float*>(p_rw), static_cast<float*>(loss.data_ptr()), grad ? grad->data_ptr() : nullptr, g.st, stream);
  if (st != SVT_OK) return PyLong_FromLong(st);
  PyObject* t = PyTuple_New(2);
  if (t == nullptr) return nullptr;
  PyTuple_SET_ITEM(t, 0, wrap(loss));
  PyTuple_SET_ITEM(t, 1, made.defined() ? wrap(made) : same(given ? a[9] : Py_None));
  return t;
}

// where(): (current device, address of its current stream, id of the capture that records the stream or 0)
PyObject* where(PyObject* const*) {
  const int device = c10::cuda::current_device();
  const auto stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
  cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
  unsigned long long id = 0;
  // (the legacy stream cannot be captured)
  if (stream != nullptr && cudaStreamGetCaptureInfo(stream, &status, &id) != cudaSuccess) {
    (void)cudaGetLastError();
    status = cudaStreamCaptureStatusNone;
  }
  return Py_BuildValue("(iKK)", device, static_cast<unsigned long long>(reinterpret_cast<uintptr_t>(stream)),
                       status == cudaStreamCaptureStatusNone ? 0ull : id);
}

// Calls `f` with its arguments; no C++ exception leaves.
template <PyObject* (*f)(PyObject* const*), int kArgs, bool kBound = true>
PyObject* guarded(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != kArgs) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", kArgs, n);
    return nullptr;
  }
  if (kBound && g_rope == nullptr) {
    PyErr_SetString(PyExc_RuntimeError, "bind has not been called");
    return nullptr;
  }
  try {
    return f(args);
  } catch (const PyFailure&) {
    return nullptr;
  } catch (const std::exception&) {
    if (!PyErr_Occurred()) torch::translate_exception_to_python(std::current_exception());  // out of memory as torch's own
    return nullptr;
  }
}

// bind(addresses of svt_rope, svt_rope_append, svt_sparse_mla_backward_workspace_size,
//      svt_sparse_mla_backward, svt_distill_topk)
PyObject* bind(PyObject* const* a) {
  auto at = [&](int i) { return reinterpret_cast<void*>(static_cast<uintptr_t>(integer(a[i]))); };
  g_rope_append = reinterpret_cast<decltype(g_rope_append)>(at(1));
  g_backward_ws = reinterpret_cast<decltype(g_backward_ws)>(at(2));
  g_backward = reinterpret_cast<decltype(g_backward)>(at(3));
  g_distill = reinterpret_cast<decltype(g_distill)>(at(4));
  g_rope = reinterpret_cast<decltype(g_rope)>(at(0));
  Py_RETURN_NONE;
}

#define SVT_METHOD(name, f, n, bound) \
  {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<f, n, bound>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {SVT_METHOD("bind", bind, 5, false),
                         SVT_METHOD("where", where, 0, false),
                         SVT_METHOD("rope", rope, 8, true),
                         SVT_METHOD("rope_append", rope_append, 15, true),
                         SVT_METHOD("sparse_mla_backward", backward, 20, true),
                         SVT_METHOD("distill_topk", distill, 10, true),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
  PyObject* m = PyModule_Create(&module);
  // what it was compiled for: the caller compares it with what runs
  if (m != nullptr && PyModule_AddStringConstant(m, "target", SVT_BINDING_TARGET) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
