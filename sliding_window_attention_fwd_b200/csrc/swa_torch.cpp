// swa_torch.cpp -- the binding's path from torch tensors to the C ABI for the
// calls that a program makes once per layer and token (rotated append,
// shared-prefix decode, shaped scores).
//
// Checking some ten tensors and converting some 25 arguments took 7 us in
// Python and 2 us in ctypes, more than the smallest of these calls take on the
// GPU; here it takes well under 1 us.  The functions take their arguments
// positionally from the wrappers in binding.py, which hold names, defaults and
// documentation.  Only marshalling happens here: dtypes, shapes and placement
// are checked (ValueError), outputs and scratch come from torch's allocator,
// and a negative status is raised as SwaError.  init() receives the addresses
// of the library's entry points.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <sstream>
#include <stdexcept>
#include <string>

#include "swa.h"

namespace {

decltype(&swa_forward_scored) g_forward = nullptr;
decltype(&swa_backward_scored) g_backward = nullptr;
decltype(&swa_rope_append_paged) g_rope = nullptr;
decltype(&swa_decode_shared) g_shared = nullptr;
decltype(&swa_decode_shared_workspace_bytes) g_shared_bytes = nullptr;
PyObject* g_error = nullptr;  // SwaError(status, where)

struct PyErrSet {};  // a Python exception is set already

[[noreturn]] void bad(const std::string& what) { throw std::invalid_argument(what); }

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) bad(std::string(name) + ": expected a torch tensor");
  return THPVariable_Unpack(o);
}

// None, or a tensor.
const at::Tensor* maybe(PyObject* o, const char* name) {
  return o == Py_None ? nullptr : &tensor(o, name);
}

long long integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PyErrSet();
  return v;
}

int int32(PyObject* o, const char* name) {
  const long long v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) bad(std::string(name) + ": out of range");
  return (int)v;
}

float real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PyErrSet();
  return (float)v;
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw PyErrSet();
  return v != 0;
}

// A size of a tensor as the library takes it.
int size32(int64_t v, const char* name) {
  if (v > INT32_MAX) bad(std::string(name) + ": too large");
  return (int)v;
}

void need(const at::Tensor& t, const char* name, at::ScalarType dtype, at::IntArrayRef shape) {
  if (t.scalar_type() != dtype || t.sizes() != shape) {
    std::ostringstream s;
    s << name << ": expected shape " << shape << " of " << dtype << ", got " << t.sizes() << " of "
      << t.scalar_type();
    bad(s.str());
  }
}

void need_dims(const at::Tensor& t, const char* name, at::ScalarType dtype, int64_t dims) {
  if (t.scalar_type() != dtype || t.dim() != dims) {
    std::ostringstream s;
    s << name << ": expected " << dims << " dims of " << dtype << ", got " << t.sizes() << " of "
      << t.scalar_type();
    bad(s.str());
  }
}

void placed(const at::Tensor& t, const char* name, const at::Tensor& ref) {
  if (!t.is_cuda() || !t.is_contiguous())
    bad(std::string(name) + ": must be a contiguous CUDA tensor");
  if (t.device() != ref.device()) {
    std::ostringstream s;
    s << name << ": on " << t.device() << ", expected " << ref.device() << " like the queries";
    bad(s.str());
  }
}

void placed(const at::Tensor* t, const char* name, const at::Tensor& ref) {
  if (t) placed(*t, name, ref);
}

template <class T = void>
T* at_or_null(const at::Tensor* t) {
  return t ? static_cast<T*>(t->data_ptr()) : nullptr;
}

// The stream of a call: None (the device's current one), an object with a
// cuda_stream attribute, or an integer handle.
struct Stream {
  cudaStream_t raw = nullptr;
  bool own = false;  // not the current one
  Stream() = default;
  Stream(PyObject* o, c10::DeviceIndex dev) {
    if (o == Py_None) {
      raw = c10::cuda::getCurrentCUDAStream(dev).stream();
      return;
    }
    own = true;
    PyObject* attr = PyObject_GetAttrString(o, "cuda_stream");
    if (!attr) {
      PyErr_Clear();
      attr = o;
      Py_INCREF(o);
    }
    const long long v = PyLong_AsLongLong(attr);
    Py_DECREF(attr);
    if (v == -1 && PyErr_Occurred()) throw PyErrSet();
    raw = reinterpret_cast<cudaStream_t>(v);
  }
  // Uninitialised device memory that torch's allocator reuses in the order of
  // this stream.
  at::Tensor empty(at::IntArrayRef shape, at::TensorOptions options, c10::DeviceIndex dev) const {
    std::optional<c10::cuda::CUDAStreamGuard> guard;
    if (own) guard.emplace(c10::cuda::getStreamFromExternal(raw, dev));
    return at::empty(shape, options);
  }
  at::Tensor scratch(int64_t n, at::ScalarType dtype, const at::Tensor& ref) const {
    return empty({n}, ref.options().dtype(dtype), ref.get_device());
  }
};

// (for tensors that are not on a GPU, which is found out later: none)
Stream stream_of(PyObject* o, const at::Tensor& q) {
  return q.is_cuda() ? Stream(o, q.get_device()) : Stream();
}

// Result of a call: the caller's tensor, or a new one (dense, of the call's
// stream).
struct Result {
  PyObject* given;
  at::Tensor made;
  const at::Tensor* t;
  Result(PyObject* o, const char* name, const at::Tensor& like, const Stream& st) : given(o) {
    if (o == Py_None) {
      made = st.empty(like.sizes(), like.options(), like.get_device());
      t = &made;
    } else {
      t = &tensor(o, name);
    }
  }
  PyObject* release() const {
    if (given == Py_None) return THPVariable_Wrap(made);
    Py_INCREF(given);
    return given;
  }
};

void raise_status(int status, const char* where) {
  PyObject* e = PyObject_CallFunction(g_error, "is", status, where);
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw PyErrSet();
}

// Runs `call` with the GIL released, on `dev`; a status other than SWA_OK is
// raised.
template <class Call>
void run(c10::DeviceIndex dev, const char* where, Call call) {
  const c10::cuda::CUDAGuard guard(dev);
  int status;
  Py_BEGIN_ALLOW_THREADS;
  status = call();
  Py_END_ALLOW_THREADS;
  if (status != SWA_OK) raise_status(status, where);
}

// What the two shaped-score calls share.
struct Scored {
  const at::Tensor &q, &k, &v;
  const at::Tensor *slopes, *cu, *prefix;
  int B, N, H, Hkv, D;
  swa_score score;
  Scored(PyObject* oq, PyObject* ok, PyObject* ov, PyObject* softcap, PyObject* oslopes,
         PyObject* ocu, PyObject* oprefix)
      : q(tensor(oq, "q")),
        k(tensor(ok, "k")),
        v(tensor(ov, "v")),
        slopes(maybe(oslopes, "slopes")),
        cu(maybe(ocu, "cu_docs")),
        prefix(maybe(oprefix, "prefix")) {
    need_dims(q, "q", at::kBFloat16, 4);
    need_dims(k, "k", at::kBFloat16, 4);
    const int64_t b = q.size(0), n = q.size(1), hkv = k.size(2), d = q.size(3);
    need(k, "k", at::kBFloat16, {b, n, hkv, d});
    need(v, "v", at::kBFloat16, {b, n, hkv, d});
    B = size32(b, "q");
    N = size32(n, "q");
    H = size32(q.size(2), "q");
    Hkv = size32(hkv, "k");
    D = size32(d, "q");
    int64_t docs = 0;
    if (slopes) need(*slopes, "slopes", at::kFloat, {q.size(2)});
    if (cu) {
      need_dims(*cu, "cu_docs", at::kInt, 2);
      docs = cu->size(1) - 1;
      if (cu->size(0) != b || docs < 1) bad("cu_docs: expected [batch, documents + 1]");
    }
    if (prefix) {
      if (!cu) bad("prefix needs cu_docs");
      need(*prefix, "prefix", at::kInt, {b, docs});
    }
    score.softcap = real(softcap);
    score.slopes = at_or_null<const float>(slopes);
    score.cu_docs = at_or_null<const int32_t>(cu);
    score.prefix = at_or_null<const int32_t>(prefix);
    score.n_docs = size32(docs, "cu_docs");
  }
  void need_lse(const at::Tensor& lse) const { need(lse, "lse", at::kFloat, {B, H, N}); }
  // (once every shape is known to be right)
  void check_placement() const {
    placed(q, "q", q);
    placed(k, "k", q);
    placed(v, "v", q);
    placed(slopes, "slopes", q);
    placed(cu, "cu_docs", q);
    placed(prefix, "prefix", q);
  }
  bool empty() const { return B == 0 || N == 0; }  // (no address to check)
};

// (q, k, v, out, lse, win_left, win_right, softcap, slopes, cu_docs, prefix,
// scale, stream) -> out
PyObject* forward_scored(PyObject* const* a) {
  const Scored s(a[0], a[1], a[2], a[7], a[8], a[9], a[10]);
  const Stream st = stream_of(a[12], s.q);
  const Result out(a[3], "out", s.q, st);
  need(*out.t, "out", at::kBFloat16, s.q.sizes());
  const at::Tensor* lse = maybe(a[4], "lse");
  if (lse) s.need_lse(*lse);
  s.check_placement();
  placed(*out.t, "out", s.q);
  placed(lse, "lse", s.q);
  const int left = int32(a[5], "win_left"), right = int32(a[6], "win_right");
  const float scale = real(a[11]);
  if (!s.empty()) {
    run(s.q.get_device(), "swa_forward_scored", [&] {
      return g_forward(s.q.data_ptr(), s.k.data_ptr(), s.v.data_ptr(), out.t->data_ptr(),
                       at_or_null<float>(lse), s.B, s.H, s.Hkv, s.N, s.D, left, right, &s.score,
                       scale, st.raw);
    });
  }
  return out.release();
}

// (q, k, v, out, dout, lse, win_left, win_right, softcap, slopes, cu_docs,
// prefix, scale, dq, dk, dv, stream) -> (dq, dk, dv)
PyObject* backward_scored(PyObject* const* a) {
  if (a[3] == Py_None || a[5] == Py_None) bad("out and lse (from the forward) are required");
  const Scored s(a[0], a[1], a[2], a[8], a[9], a[10], a[11]);
  const at::Tensor &out = tensor(a[3], "out"), &dout = tensor(a[4], "dout"),
                   &lse = tensor(a[5], "lse");
  const Stream st = stream_of(a[16], s.q);
  const Result dq(a[13], "dq", s.q, st), dk(a[14], "dk", s.k, st), dv(a[15], "dv", s.v, st);
  const struct {
    const at::Tensor& t;
    const char* name;
    const at::Tensor& like;
  } all[] = {{out, "out", s.q},   {dout, "dout", s.q}, {*dq.t, "dq", s.q},
             {*dk.t, "dk", s.k}, {*dv.t, "dv", s.k}};
  s.need_lse(lse);
  for (const auto& x : all) need(x.t, x.name, at::kBFloat16, x.like.sizes());
  s.check_placement();
  placed(lse, "lse", s.q);
  for (const auto& x : all) placed(x.t, x.name, s.q);
  const int left = int32(a[6], "win_left"), right = int32(a[7], "win_right");
  const float scale = real(a[12]);
  if (!s.empty()) {
    const at::Tensor delta = st.scratch((int64_t)s.B * s.H * s.N, at::kFloat, s.q);
    run(s.q.get_device(), "swa_backward_scored", [&] {
      return g_backward(s.q.data_ptr(), s.k.data_ptr(), s.v.data_ptr(), out.data_ptr(),
                        dout.data_ptr(), static_cast<const float*>(lse.data_ptr()),
                        dq.t->data_ptr(), dk.t->data_ptr(), dv.t->data_ptr(),
                        static_cast<float*>(delta.data_ptr()), s.B, s.H, s.Hkv, s.N, s.D, left,
                        right, &s.score, scale, st.raw);
    });
  }
  PyObject *x = dq.release(), *y = dk.release(), *z = dv.release();
  return Py_BuildValue("(NNN)", x, y, z);
}

// t [T, heads, D]: dense rows, any stride between tokens -> that stride.
int64_t token_rows(const at::Tensor& t, const char* name, const at::Tensor& ref) {
  const auto shape = t.sizes(), stride = t.strides();
  if (!t.is_cuda() || t.device() != ref.device())
    bad(std::string(name) + ": must be a CUDA tensor on the queries' device");
  if ((stride[2] != 1 && shape[2] > 1) || (stride[1] != shape[2] && shape[1] > 1))
    bad(std::string(name) + ": the rows of a token must be contiguous");
  if (shape[0] <= 1) return shape[1] * shape[2];
  if (stride[0] < shape[1] * shape[2]) bad(std::string(name) + ": tokens overlap");
  return stride[0];
}

// What the two paged calls share: the page pool.
void check_pages(const at::Tensor& kp, const at::Tensor& vp, int64_t D, int64_t page_size) {
  need_dims(kp, "k_pages", at::kBFloat16, 3);
  need(vp, "v_pages", at::kBFloat16, kp.sizes());
  if (kp.size(2) != D || page_size < 1 || kp.size(0) % page_size != 0)
    bad("k_pages, v_pages: expected [num_pages * page_size, Hkv, D]");
}

// (q, k, v, inv_freq, cu, pos0, block_table, k_pages, v_pages, page_size,
// q_out, interleaved, stream) -> q_out
PyObject* rope_append_paged(PyObject* const* a) {
  const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v"),
                   &inv = tensor(a[3], "inv_freq"), &cu = tensor(a[4], "cu"),
                   &pos0 = tensor(a[5], "pos0"), &table = tensor(a[6], "block_table"),
                   &kp = tensor(a[7], "k_pages"), &vp = tensor(a[8], "v_pages");
  const int page_size = int32(a[9], "page_size");
  need_dims(q, "q", at::kBFloat16, 3);
  const int64_t T = q.size(0), H = q.size(1), D = q.size(2);
  check_pages(kp, vp, D, page_size);
  const int64_t rows = kp.size(0), Hkv = kp.size(1);
  need(k, "k", at::kBFloat16, {T, Hkv, D});
  need(v, "v", at::kBFloat16, {T, Hkv, D});
  need_dims(inv, "inv_freq", at::kFloat, 1);
  need_dims(table, "block_table", at::kInt, 2);
  const int64_t B = table.size(0);
  need(cu, "cu", at::kInt, {B + 1});
  need(pos0, "pos0", at::kLong, {B});
  const Stream st = stream_of(a[12], q);
  const Result out(a[10], "q_out", q, st);
  need(*out.t, "q_out", at::kBFloat16, {T, H, D});
  const int64_t sq = token_rows(q, "q", q), sk = token_rows(k, "k", q), sv = token_rows(v, "v", q),
                so = token_rows(*out.t, "q_out", q);
  placed(inv, "inv_freq", q);
  placed(cu, "cu", q);
  placed(pos0, "pos0", q);
  placed(table, "block_table", q);
  placed(kp, "k_pages", q);
  placed(vp, "v_pages", q);
  const int inter = truth(a[11]);
  const int t32 = size32(T, "q"), b32 = size32(B, "block_table"), h32 = size32(H, "q"),
            kv32 = size32(Hkv, "k"), d32 = size32(D, "q"),
            pages = size32(rows / page_size, "k_pages"),
            columns = size32(table.size(1), "block_table"),
            rot = size32(2 * inv.size(0), "inv_freq");
  if (T > 0 && B > 0) {
    run(q.get_device(), "swa_rope_append_paged", [&] {
      return g_rope(q.data_ptr(), k.data_ptr(), v.data_ptr(), sq, sk, sv,
                    static_cast<const float*>(inv.data_ptr()), rot, inter,
                    static_cast<const int32_t*>(cu.data_ptr()),
                    static_cast<const int64_t*>(pos0.data_ptr()),
                    static_cast<const int32_t*>(table.data_ptr()), out.t->data_ptr(), so,
                    kp.data_ptr(), vp.data_ptr(), t32, b32, h32, kv32, d32, page_size, pages,
                    columns, st.raw);
    });
  }
  return out.release();
}

// (q, k_pages, v_pages, prefix_table, n_prefix, block_table, pos, page_size, W,
// out, lse, keep_prefix, max_tail, softcap, slopes, scale, stream) -> out
PyObject* decode_shared(PyObject* const* a) {
  const at::Tensor &q = tensor(a[0], "q"), &kp = tensor(a[1], "k_pages"),
                   &vp = tensor(a[2], "v_pages"), &ptab = tensor(a[3], "prefix_table"),
                   &table = tensor(a[5], "block_table"), &pos = tensor(a[6], "pos");
  const int n_prefix = int32(a[4], "n_prefix"), page_size = int32(a[7], "page_size"),
            W = int32(a[8], "W");
  need_dims(q, "q", at::kBFloat16, 3);
  const int64_t B = q.size(0), H = q.size(1), D = q.size(2);
  check_pages(kp, vp, D, page_size);
  need_dims(ptab, "prefix_table", at::kInt, 1);
  need_dims(table, "block_table", at::kInt, 2);
  if (table.size(0) != B) bad("block_table: expected [batch, pages]");
  need(pos, "pos", at::kLong, {B});
  if (n_prefix < 0 || ptab.size(0) * page_size < n_prefix)
    bad("prefix_table: expected the pages of n_prefix >= 0 positions");
  const Stream st = stream_of(a[16], q);
  const Result out(a[9], "out", q, st);
  need(*out.t, "out", at::kBFloat16, {B, H, D});
  const at::Tensor *lse = maybe(a[10], "lse"), *slopes = maybe(a[14], "slopes");
  if (lse) need(*lse, "lse", at::kFloat, {B, H});
  if (slopes) need(*slopes, "slopes", at::kFloat, {H});
  placed(q, "q", q);
  placed(kp, "k_pages", q);
  placed(vp, "v_pages", q);
  placed(ptab, "prefix_table", q);
  placed(table, "block_table", q);
  placed(pos, "pos", q);
  placed(*out.t, "out", q);
  placed(lse, "lse", q);
  placed(slopes, "slopes", q);
  const int keep = truth(a[11]);
  const float softcap = real(a[13]), scale = real(a[15]);
  long long tail = a[12] == Py_None ? table.size(1) * (long long)page_size - n_prefix
                                    : integer(a[12]);
  tail = tail < 0 ? 0 : (tail > INT32_MAX ? INT32_MAX : tail);
  const int b32 = size32(B, "q"), h32 = size32(H, "q"), kv32 = size32(kp.size(1), "k_pages"),
            d32 = size32(D, "q"), pages = size32(kp.size(0) / page_size, "k_pages"),
            columns = size32(table.size(1), "block_table");
  if (B > 0) {
    const auto dev = q.get_device();
    size_t bytes;
    {
      const c10::cuda::CUDAGuard guard(dev);
      bytes = g_shared_bytes(b32, h32, kv32, d32, n_prefix, W, (int)tail);
    }
    const at::Tensor ws = st.scratch(bytes < 16 ? 16 : (int64_t)bytes, at::kByte, q);
    run(dev, "swa_decode_shared", [&] {
      return g_shared(q.data_ptr(), kp.data_ptr(), vp.data_ptr(), out.t->data_ptr(),
                      at_or_null<float>(lse),
                      n_prefix ? static_cast<const int32_t*>(ptab.data_ptr()) : nullptr, n_prefix,
                      static_cast<const int32_t*>(table.data_ptr()),
                      static_cast<const int64_t*>(pos.data_ptr()), b32, h32, kv32, d32, page_size,
                      pages, columns, W, keep, (int)tail, softcap,
                      at_or_null<const float>(slopes), scale, ws.data_ptr(), ws.numel(), st.raw);
    });
  }
  return out.release();
}

// Argument count, and no C++ exception past this point.
template <PyObject* (*kCall)(PyObject* const*), int kArgs>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != kArgs) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return kCall(args);
  } catch (const PyErrSet&) {
  } catch (const std::invalid_argument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// (SwaError, addresses of swa_forward_scored, swa_backward_scored,
// swa_rope_append_paged, swa_decode_shared, swa_decode_shared_workspace_bytes)
PyObject* init(PyObject* const* a) {
  Py_INCREF(a[0]);
  Py_XSETREF(g_error, a[0]);
  g_forward = reinterpret_cast<decltype(g_forward)>(integer(a[1]));
  g_backward = reinterpret_cast<decltype(g_backward)>(integer(a[2]));
  g_rope = reinterpret_cast<decltype(g_rope)>(integer(a[3]));
  g_shared = reinterpret_cast<decltype(g_shared)>(integer(a[4]));
  g_shared_bytes = reinterpret_cast<decltype(g_shared_bytes)>(integer(a[5]));
  Py_RETURN_NONE;
}

template <PyObject* (*kCall)(PyObject* const*), int kArgs>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<kCall, kArgs>)),
          METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {
    method<init, 6>("init"),
    method<forward_scored, 13>("forward_scored"),
    method<backward_scored, 17>("backward_scored"),
    method<rope_append_paged, 13>("rope_append_paged"),
    method<decode_shared, 17>("decode_shared"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, g_methods};

}  // namespace

PyMODINIT_FUNC PyInit__torch_calls() { return PyModule_Create(&g_module); }
