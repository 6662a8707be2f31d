// serving_binding.cpp - the serving operators' Python entry points: checks torch tensors,
// allocates the outputs that are not given and calls the C ABI of libattn on the tensors'
// device and stream.
//
// A decode step's kernels take a few microseconds each, so what a call costs on the host
// counts: marshalled in Python a call took 20 microseconds and more, from here about six.
// Positional arguments only; serving.py has the signatures, defaults and documentation.
#include <ATen/cuda/EmptyTensor.h>
#include <Python.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "../../include/attn.h"

namespace {

using at::ScalarType;

PyObject* g_attn_error = nullptr;  // AttnError(status, where)

[[noreturn]] void refuse(const std::string& what) {
  PyErr_SetString(PyExc_ValueError, what.c_str());
  throw python_error();
}

std::string text(at::IntArrayRef s) {
  std::string r = "[";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + "]";
}

const at::Tensor& cuda_tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda())
    refuse(std::string(name) + " must be a CUDA tensor");
  return THPVariable_Unpack(o);
}

void need_type(const at::Tensor& t, ScalarType type, const char* name) {
  if (t.scalar_type() != type)
    refuse(std::string(name) + " must be " + c10::toString(type) + ", got " +
           c10::toString(t.scalar_type()));
}

// A tensor whose shape the others follow.
const at::Tensor& lead(PyObject* o, ScalarType type, int64_t dims, const char* name) {
  const at::Tensor& t = cuda_tensor(o, name);
  need_type(t, type, name);
  if (t.dim() != dims)
    refuse(std::string(name) + " must have " + std::to_string(dims) + " dimensions, got " +
           text(t.sizes()));
  if (t.numel() == 0) refuse(std::string(name) + " must not be empty, got " + text(t.sizes()));
  return t;
}

// The address of a contiguous tensor of this type, shape and device.
void* address(const at::Tensor& t, ScalarType type, at::IntArrayRef shape, c10::Device dev,
              const char* name) {
  need_type(t, type, name);
  if (t.sizes() != shape)
    refuse(std::string(name) + " must be " + text(shape) + ", got " + text(t.sizes()));
  if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
  if (t.device() != dev)
    refuse(std::string(name) + " must be on " + dev.str() + ", got " + t.device().str());
  return t.data_ptr();
}

void* address(PyObject* o, ScalarType type, at::IntArrayRef shape, c10::Device dev,
              const char* name) {
  return address(cuda_tensor(o, name), type, shape, dev, name);
}

// A piece of a buffer as a tensor of its own: several small outputs of one allocation (an
// allocation costs more than all the rest of a small call's marshalling).
at::Tensor piece(const at::Tensor& buf, int64_t* at, at::IntArrayRef shape) {
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::TensorImpl::VIEW,
                                                         c10::Storage(buf.storage()), buf.key_set(),
                                                         buf.dtype());
  c10::TensorImpl* impl = t.unsafeGetTensorImpl();
  impl->set_storage_offset(*at);
  impl->set_sizes_contiguous(shape);
  *at += c10::multiply_integers(shape);
  return t;
}

long long integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}

int integer32(PyObject* o, const char* name) {
  const long long v = integer(o);
  if (v > INT32_MAX || v < INT32_MIN) refuse(std::string(name) + " does not fit 32 bits");
  return static_cast<int>(v);
}

double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}

int size32(int64_t v, const char* name) {
  if (v > INT32_MAX) refuse(std::string(name) + " is too large");
  return static_cast<int>(v);
}

// Where a call runs: its device, and the given stream (a handle, an integer) or the device's
// current one. While it lives that stream is the current one, so what the call allocates comes
// from its pool: a block that was freed on the caller's stream may still be in use there.
class Launch {
 public:
  Launch(PyObject* o, c10::Device dev)
      : dev_(dev), caller_(c10::cuda::getCurrentCUDAStream(dev.index())), stream_(pick(o)) {
    if (o == Py_None)
      device_.set_device(dev);
    else
      given_.reset_stream(stream_);
  }

  void* stream() const { return stream_.stream(); }

  // Memory for this call alone.
  at::Tensor scratch(int64_t bytes) const { return empty({bytes}, ScalarType::Byte); }

  // An output: the caller's stream is likely to use it next, and to be where it is dropped.
  at::Tensor fresh(at::IntArrayRef shape, ScalarType type) const {
    at::Tensor t = empty(shape, type);
    if (stream_ != caller_) t.record_stream(caller_);
    return t;
  }

  // The given output, checked, or a new one.
  at::Tensor output(PyObject* o, at::IntArrayRef shape, ScalarType type, const char* name) const {
    if (o == Py_None) return fresh(shape, type);
    const at::Tensor& t = cuda_tensor(o, name);
    address(t, type, shape, dev_, name);
    return t;
  }

 private:
  at::Tensor empty(at::IntArrayRef shape, ScalarType type) const {
    return at::detail::empty_cuda(shape, type, dev_, std::nullopt);
  }
  c10::cuda::CUDAStream pick(PyObject* o) const {
    if (o == Py_None) return caller_;
    auto s = reinterpret_cast<cudaStream_t>(integer(o));
    if (s == cudaStreamLegacy) s = nullptr;  // the default stream has both names
    return c10::cuda::getStreamFromExternal(s, dev_.index());
  }

  c10::Device dev_;
  c10::cuda::CUDAStream caller_, stream_;
  // one of the two (the stream's sets the device too, and costs 0.1 us more)
  c10::cuda::OptionalCUDAGuard device_;
  c10::cuda::OptionalCUDAStreamGuard given_;
};

void check(attn_status_t st, const char* where) {
  if (st == ATTN_OK) return;
  PyObject* e = PyObject_CallFunction(g_attn_error, "is", static_cast<int>(st), where);
  if (e) {
    PyErr_SetObject(g_attn_error, e);
    Py_DECREF(e);
  }
  throw python_error();
}

template <class... T>
PyObject* pack(const T&... t) {
  PyObject* r = PyTuple_New(sizeof...(T));
  if (!r) throw python_error();
  Py_ssize_t i = 0;
  (PyTuple_SET_ITEM(r, i++, THPVariable_Wrap(t)), ...);
  return r;
}

struct Cache {
  void* p;
  int n_pages, Hkv, page, d;
};

Cache cache_of(PyObject* o, c10::Device dev) {
  const at::Tensor& t = cuda_tensor(o, "cache");
  if (t.scalar_type() != ScalarType::Byte || t.dim() != 4 || (t.size(3) != 1280 && t.size(3) != 2560))
    refuse("cache must be uint8 [n_pages, Hkv, page_size / 16, 20 d], d 64 or 128");
  if (!t.is_contiguous() || t.numel() == 0) refuse("cache must be contiguous and not empty");
  if (t.device() != dev) refuse("cache must be on " + dev.str() + ", got " + t.device().str());
  if (t.size(2) > INT32_MAX / 16) refuse("cache pages are too large");
  return Cache{t.data_ptr(), size32(t.size(0), "n_pages"), size32(t.size(1), "Hkv"),
               static_cast<int>(t.size(2)) * 16, static_cast<int>(t.size(3)) / 20};
}

const at::Tensor& table_of(PyObject* o, int64_t B, c10::Device dev) {
  const at::Tensor& t = lead(o, ScalarType::Int, 2, "table");
  if (t.device() != dev || t.size(0) != B)
    refuse("table must be [" + std::to_string(B) + ", width] on " + dev.str());
  return t;
}

#define OSX_ENTRY(name, count)                                               \
  PyObject* name(PyObject*, PyObject* const* a, Py_ssize_t n) {              \
    HANDLE_TH_ERRORS                                                         \
    if (n != count) {                                                        \
      PyErr_SetString(PyExc_TypeError, #name " takes " #count " arguments"); \
      return nullptr;                                                        \
    }
#define OSX_END       \
  END_HANDLE_TH_ERRORS \
  }

// lens, new_lens, table, free_pages, free_head, page_size, n_new, stream
OSX_ENTRY(kv_plan, 8)
  const at::Tensor& lens = lead(a[0], ScalarType::Int, 1, "lens");
  const c10::Device dev = lens.device();
  const int64_t B = lens.size(0);
  const at::Tensor& table = table_of(a[2], B, dev);
  const at::Tensor& free_pages = cuda_tensor(a[3], "free_pages");
  if (free_pages.dim() != 1) refuse("free_pages must be one-dimensional");
  const int page = integer32(a[5], "page_size"), n_new = integer32(a[6], "n_new");
  if (n_new < 1 || page < 1) refuse("need n_new >= 1 and page_size >= 1");
  const auto* lens_p = static_cast<int32_t*>(address(lens, ScalarType::Int, {B}, dev, "lens"));
  const auto* new_p = static_cast<int32_t*>(address(a[1], ScalarType::Int, {B}, dev, "new_lens"));
  auto* table_p = static_cast<int32_t*>(address(table, ScalarType::Int, table.sizes(), dev, "table"));
  const auto* free_p = static_cast<int32_t*>(
      address(free_pages, ScalarType::Int, free_pages.sizes(), dev, "free_pages"));
  const auto* head_p = static_cast<int32_t*>(address(a[4], ScalarType::Int, {1}, dev, "free_head"));
  const Launch run(a[7], dev);
  const at::Tensor buf = run.fresh({2 * B * n_new + 2 * B + 1}, ScalarType::Int);
  int64_t at = 0;
  at::Tensor slots = piece(buf, &at, {B, n_new}), pos = piece(buf, &at, {B, n_new});
  at::Tensor out = piece(buf, &at, {B}), served = piece(buf, &at, {B}), head = piece(buf, &at, {1});
  // an empty list has no address of its own
  check(attn_kv_plan(lens_p, new_p, table_p, free_p ? free_p : lens_p, head_p,
                     static_cast<int32_t*>(slots.data_ptr()), static_cast<int32_t*>(pos.data_ptr()),
                     static_cast<int32_t*>(out.data_ptr()), static_cast<int32_t*>(head.data_ptr()),
                     static_cast<int32_t*>(served.data_ptr()), size32(B, "B"), n_new,
                     size32(table.size(1), "width"), page, size32(free_pages.size(0), "free_pages"),
                     run.stream()),
        "attn_kv_plan");
  return pack(slots, pos, out, head, served);
OSX_END

// qkv, wq, wk, inv_freq, positions, n_heads, n_kv_heads, eps, interleaved, q, k, v, stream
OSX_ENTRY(qk_norm_rope, 13)
  const at::Tensor& qkv = lead(a[0], ScalarType::BFloat16, 3, "qkv");
  const c10::Device dev = qkv.device();
  const int64_t B = qkv.size(0), N = qkv.size(1), width = qkv.size(2);
  const int Hq = integer32(a[5], "n_heads"), Hkv = integer32(a[6], "n_kv_heads");
  if (Hq < 1 || Hkv < 1) refuse("need n_heads, n_kv_heads >= 1");
  const int64_t H = Hq + 2ll * Hkv, d = width / H;
  if (width != H * d || (d != 64 && d != 128))
    refuse("qkv's last dimension must be (n_heads + 2 n_kv_heads) d, d 64 or 128");
  if (qkv.stride(2) != 1) refuse("qkv's last dimension must be contiguous");
  const at::Tensor& wq = cuda_tensor(a[1], "wq");
  if (wq.scalar_type() != ScalarType::BFloat16 && wq.scalar_type() != ScalarType::Float)
    refuse("wq and wk must be bf16 or fp32 tensors");
  const at::Tensor& inv = cuda_tensor(a[3], "inv_freq");
  if (inv.dim() != 1 || inv.size(0) < 1 || 2 * inv.size(0) > d)
    refuse("inv_freq must be fp32 [r / 2] with 0 < r <= d");
  const void* wq_p = address(wq, wq.scalar_type(), {d}, dev, "wq");
  const void* wk_p = address(a[2], wq.scalar_type(), {d}, dev, "wk");
  const auto* f_p = static_cast<float*>(address(inv, ScalarType::Float, inv.sizes(), dev, "inv_freq"));
  const auto* p_p = static_cast<int32_t*>(address(a[4], ScalarType::Int, {B, N}, dev, "positions"));
  const int inter = PyObject_IsTrue(a[8]);
  if (inter < 0) throw python_error();
  const Launch run(a[12], dev);
  at::Tensor q = run.output(a[9], {B, Hq, N, d}, ScalarType::BFloat16, "q");
  at::Tensor k = run.output(a[10], {B, Hkv, N, d}, ScalarType::BFloat16, "k");
  at::Tensor v = run.output(a[11], {B, Hkv, N, d}, ScalarType::BFloat16, "v");
  // the stride of a dimension of one row is never used
  check(attn_qk_norm_rope(qkv.data_ptr(), B > 1 ? qkv.stride(0) : 0, N > 1 ? qkv.stride(1) : 0, wq_p,
                          wk_p, wq.scalar_type() == ScalarType::Float, f_p,
                          static_cast<int>(inv.size(0)), p_p, q.data_ptr(), k.data_ptr(),
                          v.data_ptr(), size32(B, "B"), size32(N, "N"), Hq, Hkv,
                          static_cast<int>(d), static_cast<float>(real(a[7])), inter,
                          run.stream()),
        "attn_qk_norm_rope");
  return pack(q, k, v);
OSX_END

// k, v, cache, slots, stream
OSX_ENTRY(kv4_append, 5)
  const at::Tensor& k = lead(a[0], ScalarType::BFloat16, 4, "k");
  const c10::Device dev = k.device();
  const Cache c = cache_of(a[2], dev);
  const int64_t B = k.size(0), N = k.size(2);
  if (k.size(1) != c.Hkv || k.size(3) != c.d)
    refuse("k must be [B, " + std::to_string(c.Hkv) + ", N, " + std::to_string(c.d) +
           "] as the cache is, got " + text(k.sizes()));
  const void* k_p = address(k, ScalarType::BFloat16, k.sizes(), dev, "k");
  const void* v_p = address(a[1], ScalarType::BFloat16, k.sizes(), dev, "v");
  const auto* s_p = static_cast<int32_t*>(address(a[3], ScalarType::Int, {B, N}, dev, "slots"));
  const Launch run(a[4], dev);
  check(attn_kv4_append(k_p, v_p, c.p, s_p, size32(B, "B"), c.Hkv, size32(N, "N"), c.d, c.page,
                        c.n_pages, run.stream()),
        "attn_kv4_append");
  Py_RETURN_NONE;
OSX_END

// cache, table, start, lens, n, k, v, stream
OSX_ENTRY(kv4_read, 8)
  const at::Tensor& table = lead(a[1], ScalarType::Int, 2, "table");
  const c10::Device dev = table.device();
  const Cache c = cache_of(a[0], dev);
  const int64_t B = table.size(0);
  const int n_tok = integer32(a[4], "n");
  if (n_tok < 1) refuse("need n >= 1");
  const auto* t_p = static_cast<int32_t*>(address(table, ScalarType::Int, table.sizes(), dev, "table"));
  const auto* s_p = static_cast<int32_t*>(address(a[2], ScalarType::Int, {B}, dev, "start"));
  const auto* l_p = static_cast<int32_t*>(address(a[3], ScalarType::Int, {B}, dev, "lens"));
  const Launch run(a[7], dev);
  at::Tensor k = run.output(a[5], {B, c.Hkv, n_tok, c.d}, ScalarType::BFloat16, "k");
  at::Tensor v = run.output(a[6], {B, c.Hkv, n_tok, c.d}, ScalarType::BFloat16, "v");
  check(attn_kv4_read(c.p, t_p, s_p, l_p, k.data_ptr(), v.data_ptr(), size32(B, "B"), c.Hkv, n_tok,
                      c.d, c.page, c.n_pages, size32(table.size(1), "width"), run.stream()),
        "attn_kv4_read");
  return pack(k, v);
OSX_END

// The output rows' type: that of the given output, or of the flag.
ScalarType o_type(PyObject* o, PyObject* bf16) {
  if (o == Py_None) {
    const int b = PyObject_IsTrue(bf16);
    if (b < 0) throw python_error();
    return b ? ScalarType::BFloat16 : ScalarType::Float;
  }
  const ScalarType t = cuda_tensor(o, "o").scalar_type();
  if (t != ScalarType::BFloat16 && t != ScalarType::Float) refuse("o must be fp32 or bf16");
  return t;
}

// q, cache, table, lens, q_pos, window, sinks, scale, max_len, bf16, o, lse, stream
OSX_ENTRY(kv4_fwd, 13)
  const at::Tensor& q = lead(a[0], ScalarType::BFloat16, 4, "q");
  const c10::Device dev = q.device();
  const Cache c = cache_of(a[1], dev);
  const int64_t B = q.size(0), Hq = q.size(1), Nq = q.size(2), d = q.size(3);
  if (d != c.d || Hq % c.Hkv)
    refuse("q must be [B, Hq, Nq, " + std::to_string(c.d) + "] with Hq a multiple of " +
           std::to_string(c.Hkv) + ", got " + text(q.sizes()));
  const at::Tensor& table = table_of(a[2], B, dev);
  const void* q_p = address(q, ScalarType::BFloat16, q.sizes(), dev, "q");
  const auto* t_p = static_cast<int32_t*>(address(table, ScalarType::Int, table.sizes(), dev, "table"));
  const auto* l_p = static_cast<int32_t*>(address(a[3], ScalarType::Int, {B}, dev, "lens"));
  const auto* p_p = a[4] == Py_None
                        ? nullptr
                        : static_cast<int32_t*>(address(a[4], ScalarType::Int, {B}, dev, "q_pos"));
  const ScalarType type = o_type(a[10], a[9]);
  const Launch run(a[12], dev);
  at::Tensor o = run.output(a[10], {B, Hq, Nq, d}, type, "o");
  at::Tensor lse = run.output(a[11], {B, Hq, Nq}, ScalarType::Float, "lse");
  const int b = size32(B, "B"), hq = size32(Hq, "Hq"), nq = size32(Nq, "Nq");
  const int64_t n_ws = attn_kv4_fwd_workspace(b, hq, c.Hkv, nq, c.d);
  at::Tensor ws = run.scratch(n_ws);
  check(attn_kv4_fwd(q_p, c.p, t_p, l_p, p_p, o.data_ptr(), static_cast<float*>(lse.data_ptr()),
                     type == ScalarType::BFloat16, b, hq, c.Hkv, nq, c.d, c.page, c.n_pages,
                     size32(table.size(1), "width"), integer(a[8]), integer32(a[5], "window"),
                     integer32(a[6], "sinks"), static_cast<float>(real(a[7])), ws.data_ptr(), n_ws,
                     run.stream()),
        "attn_kv4_fwd");
  return pack(o, lse);
OSX_END

// q, k, v, window, sinks, q_off, kv_off, kv_len, scale, bf16, o, lse, stream
OSX_ENTRY(window_fwd, 13)
  const at::Tensor& q = lead(a[0], ScalarType::BFloat16, 4, "q");
  const c10::Device dev = q.device();
  const int64_t B = q.size(0), Hq = q.size(1), Nq = q.size(2), d = q.size(3);
  const at::Tensor& k = lead(a[1], ScalarType::BFloat16, 4, "k");
  if (k.device() != dev || k.size(0) != B || k.size(3) != d)
    refuse("k and v must be [" + std::to_string(B) + ", Hkv, L, " + std::to_string(d) + "] on " +
           dev.str());
  const int64_t Hkv = k.size(1), L = k.size(2);
  const int64_t n_keys = a[7] == Py_None ? L : integer(a[7]);
  if (n_keys < 1 || n_keys > L) refuse("kv_len must be in 1.." + std::to_string(L));
  const int64_t kv_off = integer(a[6]);
  int64_t q_off;
  if (a[5] == Py_None) {
    q_off = kv_off + n_keys - Nq;
    if (q_off < 0) refuse("more query rows than key rows: give q_off");
  } else {
    q_off = integer(a[5]);
  }
  const void* q_p = address(q, ScalarType::BFloat16, q.sizes(), dev, "q");
  const void* k_p = address(k, ScalarType::BFloat16, k.sizes(), dev, "k");
  const void* v_p = address(a[2], ScalarType::BFloat16, k.sizes(), dev, "v");
  const ScalarType type = o_type(a[10], a[9]);
  const Launch run(a[12], dev);
  at::Tensor o = run.output(a[10], {B, Hq, Nq, d}, type, "o");
  at::Tensor lse = run.output(a[11], {B, Hq, Nq}, ScalarType::Float, "lse");
  const int b = size32(B, "B"), hq = size32(Hq, "Hq"), hkv = size32(Hkv, "Hkv");
  const int64_t n_ws = attn_window_fwd_workspace(b, hq, hkv, Nq, static_cast<int>(d));
  at::Tensor ws;
  if (n_ws > 0) ws = run.scratch(n_ws);
  check(attn_window_fwd(q_p, k_p, v_p, o.data_ptr(), static_cast<float*>(lse.data_ptr()),
                        type == ScalarType::BFloat16, b, hq, hkv, Nq, n_keys, Nq, L, q_off, kv_off,
                        size32(d, "d"), integer32(a[3], "window"), integer32(a[4], "sinks"),
                        static_cast<float>(real(a[8])), n_ws > 0 ? ws.data_ptr() : nullptr, n_ws,
                        run.stream()),
        "attn_window_fwd");
  return pack(o, lse);
OSX_END

// the exception class that carries a status
PyObject* set_error(PyObject*, PyObject* cls) {
  Py_XDECREF(g_attn_error);
  Py_INCREF(cls);
  g_attn_error = cls;
  Py_RETURN_NONE;
}

#define OSX_METHOD(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {OSX_METHOD(kv_plan),    OSX_METHOD(qk_norm_rope), OSX_METHOD(kv4_append),
                           OSX_METHOD(kv4_read),   OSX_METHOD(kv4_fwd),      OSX_METHOD(window_fwd),
                           {"set_error", set_error, METH_O, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_serving", nullptr, -1, g_methods,
                        nullptr,               nullptr,    nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serving(void) {
  PyObject* m = PyModule_Create(&g_module);
  // (the versions that the build compiled against; the loader compares them)
  if (m && PyModule_AddStringConstant(m, "built_for", OSX_BUILT_FOR) < 0) Py_CLEAR(m);
  return m;
}
