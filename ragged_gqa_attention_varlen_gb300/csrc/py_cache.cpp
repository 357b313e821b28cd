// py_cache.cpp -- Python entry of the generation calls: checks the tensors,
// allocates what the caller did not pass and calls the C ABI.
//
// The calls of a decode step take a few microseconds on the GPU; reading some
// sixty tensor attributes and converting forty arguments in Python took 25 to
// 40 microseconds of host time per call, so that is done here (about 5).  The
// library's functions come as addresses from the ctypes binding, which stays
// the one place that loads it.
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>
#include <ATen/ops/zeros.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <optional>
#include <stdexcept>
#include <string>
#include <vector>

#include "../../include/attn_varlen.h"

namespace {

struct Fns {
  decltype(&attn_varlen_rotary) rotary;
  decltype(&attn_varlen_cache_append) append;
  decltype(&attn_varlen_cache_fwd) fwd;
  decltype(&attn_varlen_cache_fwd_workspace_size) fwd_ws;
  decltype(&attn_varlen_cache_weights) weights;
  decltype(&attn_varlen_cache_weights_workspace_size) weights_ws;
  decltype(&attn_varlen_cache_evict) evict;
  decltype(&attn_varlen_cache_evict_workspace_size) evict_ws;
  decltype(&attn_varlen_norm_rotary) norm;
  decltype(&attn_varlen_norm_rotary_bwd) norm_bwd;
  decltype(&attn_varlen_norm_rotary_bwd_workspace_size) norm_bwd_ws;
  decltype(&attn_varlen_cache8_append) append8;
  decltype(&attn_varlen_cache8_fwd) fwd8;
  decltype(&attn_varlen_cache8_fwd_workspace_size) fwd8_ws;
  decltype(&attn_varlen_cache_fork) fork;
  decltype(&attn_varlen_cache_fork_workspace_size) fork_ws;
  decltype(&attn_varlen_cache_compact) compact;
  decltype(&attn_varlen_cache_compact_workspace_size) compact_ws;
  decltype(&attn_varlen_cache_copy) copy;
  decltype(&attn_status_string) status_string;
} fn;
PyObject* attn_error = nullptr;  // the exception of a negative status

struct Failed {
  attn_status code;
};
void check(attn_status s) {
  if (s != ATTN_OK) throw Failed{s};
}
[[noreturn]] void bad(const std::string& what) { throw std::invalid_argument(what); }

using at::Tensor;
using Maybe = const Tensor*;

Maybe maybe(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) throw std::invalid_argument(std::string(name) + " must be a tensor or None");
  return &THPVariable_Unpack(o);
}
const Tensor& tensor(PyObject* o, const char* name) {
  Maybe t = maybe(o, name);
  if (!t) bad(std::string(name) + " must be a tensor");
  return *t;
}
int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    bad("an option must be an integer");
  }
  return v;
}
int small(PyObject* o) {
  const int64_t v = integer(o);
  return static_cast<int>(v < INT32_MIN ? INT32_MIN : (v > INT32_MAX ? INT32_MAX : v));
}
double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    bad("an option must be a number");
  }
  return v;
}
struct Raised {};  // a Python error is set
int truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised{};
  return v;
}

// A call's device, made current for its duration, and its stream.
struct Call {
  c10::Device device;
  c10::cuda::OptionalCUDAGuard guard;
  explicit Call(const Tensor& first) : device(first.device()) {
    if (!first.is_cuda()) bad("the tensors of a call must be CUDA tensors");
    guard.set_device(device);
  }
  void* stream() const { return c10::cuda::getCurrentCUDAStream(device.index()).stream(); }
  const Tensor& here(const Tensor& t, const char* name) const {
    if (t.device() != device) bad(std::string(name) + " must be on the device of the call's other tensors");
    return t;
  }
  Tensor make(at::IntArrayRef shape, at::ScalarType type) const {
    return at::empty(shape, at::TensorOptions().dtype(type).device(device));
  }
};

attn_dtype dtype_of(const Tensor& t) {
  if (t.scalar_type() == at::kBFloat16) return ATTN_BF16;
  if (t.scalar_type() == at::kHalf) return ATTN_F16;
  bad("q, k, v and the cache must be fp16 or bf16");
}
bool head_dim(int64_t d) { return d == 64 || d == 128 || d == 160; }

// A stride that no index uses (an axis of one) may be anything.
int64_t used(int64_t stride, int64_t size, int64_t dense) { return size > 1 ? stride : dense; }

struct Rows {  // packed [tokens, heads, d]
  void* p = nullptr;
  int64_t ts = 0, hs = 0;
};
Rows rows16(const Call& c, const Tensor& t, const char* name, at::ScalarType type, int64_t heads,
            int64_t d, int64_t tokens) {
  c.here(t, name);
  if (t.scalar_type() != type || t.dim() != 3 || t.size(0) != tokens || t.size(1) != heads ||
      t.size(2) != d || t.stride(2) != 1)
    bad(std::string(name) + " must be [" + std::to_string(tokens) + ", " + std::to_string(heads) + ", " +
        std::to_string(d) + "] of the call's 16-bit type with a contiguous feature axis");
  return {t.data_ptr(), used(t.stride(0), tokens, heads * d), used(t.stride(1), heads, d)};
}

struct Pool {  // [num_pages, page_size, Hkv, d]
  void* p;
  int64_t ps, ss, hs;
};
Pool pool(const Call& c, const Tensor& t, const char* name, at::ScalarType type) {
  c.here(t, name);
  if (t.scalar_type() != type || t.dim() != 4 || t.stride(3) != 1 || t.size(0) > INT32_MAX ||
      t.size(1) > 1024)
    bad(std::string(name) + " must be [num_pages, page_size, Hkv, d] of " +
        (type == at::kFloat8_e4m3fn ? "float8_e4m3fn" : "the call's 16-bit type") +
        " with a contiguous feature axis and at most 1024 rows a page");
  const int64_t ps = t.size(1), h = t.size(2), d = t.size(3);
  return {t.data_ptr(), used(t.stride(0), t.size(0), ps * h * d), used(t.stride(1), ps, h * d),
          used(t.stride(2), h, d)};
}

const int32_t* vec(const Call& c, const Tensor& t, const char* name, int64_t n) {
  c.here(t, name);
  if (t.scalar_type() != at::kInt || t.dim() != 1 || t.size(0) != n || (n > 1 && t.stride(0) != 1))
    bad(std::string(name) + " must be a contiguous int32 CUDA vector of " + std::to_string(n));
  return t.data_ptr<int32_t>();
}
int32_t* status_of(const Call& c, Maybe t) {
  if (!t) return nullptr;
  c.here(*t, "status");
  if (t->scalar_type() != at::kInt || t->numel() < 1) bad("status must be an int32 CUDA tensor");
  return t->data_ptr<int32_t>();
}

struct Tab {
  const int32_t* p = nullptr;
  int64_t rs = 0;
  int width = 0;
  const int32_t* lens = nullptr;
  int64_t rows = 0;
};
Tab table(const Call& c, const Tensor& t, const Tensor& lens, const char* name) {
  c.here(t, name);
  Tab r;
  r.rows = lens.numel();
  if (t.scalar_type() != at::kInt || t.dim() != 2 || t.size(0) != r.rows || t.size(1) < 1 ||
      t.size(1) > INT32_MAX || (t.size(1) > 1 && t.stride(1) != 1))
    bad(std::string(name) + " must be an int32 CUDA tensor [" + std::to_string(r.rows) +
        ", width] with contiguous rows");
  r.p = t.data_ptr<int32_t>();
  r.width = static_cast<int>(t.size(1));
  r.rs = used(t.stride(0), r.rows, r.width);
  r.lens = vec(c, lens, "the lengths of a table", r.rows);
  return r;
}

template <class T>
struct Slots {  // [rows, Hkv, at least slots]
  T* p = nullptr;
  int64_t rs = 0, hs = 0;
};
template <class T>
Slots<T> slots(const Call& c, Maybe t, const char* name, int64_t rows, int64_t heads, int64_t n) {
  Slots<T> s;
  if (!t) return s;
  c.here(*t, name);
  if (t->scalar_type() != c10::CppTypeToScalarType<T>::value || t->dim() != 3 || t->size(0) != rows ||
      t->size(1) != heads || t->size(2) < n || (t->size(2) > 1 && t->stride(2) != 1))
    bad(std::string(name) + " must be " + (sizeof(T) == 4 && std::is_same<T, float>::value ? "fp32" : "int32") +
        " [" + std::to_string(rows) + ", " + std::to_string(heads) + ", at least " + std::to_string(n) +
        "] on the device, slots contiguous");
  s.p = t->data_ptr<T>();
  s.rs = t->stride(0);
  s.hs = t->stride(1);
  return s;
}

struct Workspace {
  Tensor own;
  void* p;
  size_t bytes;
};
Workspace workspace(const Call& c, Maybe given, size_t need) {
  Workspace w;
  if (given) {
    c.here(*given, "workspace");
    if (!given->is_contiguous()) bad("workspace must be contiguous");
    w.p = given->data_ptr();
    w.bytes = given->nbytes();
  } else {
    w.own = c.make({static_cast<int64_t>(need < 256 ? 256 : need)}, at::kByte);
    w.p = w.own.data_ptr();
    w.bytes = w.own.nbytes();
  }
  return w;
}

struct Rotary {
  const int32_t* pos = nullptr;
  int64_t axis_stride = 0;
  int axes = 1;
  const double* freq = nullptr;
  const int32_t* axis = nullptr;
  int pairs = 0;
};
Rotary rotary(const Call& c, Maybe positions, Maybe inv_freq, Maybe pair_axis, int64_t d, int64_t tokens) {
  Rotary r;
  if (!positions) {
    if (inv_freq) bad("rotary positions are missing");
    return r;
  }
  const Tensor& t = c.here(*positions, "positions");
  const bool one = t.dim() == 1;
  if (t.scalar_type() != at::kInt || (t.dim() != 1 && t.dim() != 2) || t.size(one ? 0 : 1) != tokens ||
      (!one && t.size(0) < 1) || (tokens > 1 && t.stride(one ? 0 : 1) != 1))
    bad("positions must be an int32 CUDA tensor [axes, " + std::to_string(tokens) + "] or [" +
        std::to_string(tokens) + "], rows contiguous");
  r.pos = t.data_ptr<int32_t>();
  r.axes = one ? 1 : static_cast<int>(t.size(0));
  r.axis_stride = one ? 0 : t.stride(0);
  if (!inv_freq) return r;
  c.here(*inv_freq, "inv_freq");
  const int64_t pairs = inv_freq->numel();
  if (inv_freq->scalar_type() != at::kDouble || inv_freq->dim() != 1 || !inv_freq->is_contiguous() ||
      pairs < 1 || 2 * pairs > d)
    bad("inv_freq must be a contiguous float64 CUDA vector of 1 to " + std::to_string(d / 2) + " pairs");
  r.freq = inv_freq->data_ptr<double>();
  r.pairs = static_cast<int>(pairs);
  if (pair_axis) r.axis = vec(c, *pair_axis, "pair_axis", pairs);
  return r;
}

PyObject* kept(PyObject* o) {
  Py_INCREF(o);
  return o;
}
// The caller's object, or a new tensor.
PyObject* result(PyObject* given, const Tensor& t) { return given != Py_None ? kept(given) : THPVariable_Wrap(t); }

template <class F>
PyObject* guarded(Py_ssize_t nargs, Py_ssize_t want, F f) {
  if (!fn.rotary || nargs != want) {
    PyErr_SetString(PyExc_TypeError, "internal: the library is not bound, or the argument count is wrong");
    return nullptr;
  }
  try {
    return f();
  } catch (const Failed& e) {
    PyObject* x = PyObject_CallFunction(attn_error, "is", static_cast<int>(e.code), fn.status_string(e.code));
    if (x) {
      PyErr_SetObject(attn_error, x);
      Py_DECREF(x);
    }
  } catch (const std::invalid_argument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const Raised&) {
  } catch (const python_error&) {
    // (its Python error is set)
  } catch (const c10::OutOfMemoryError& e) {
    PyObject* torch = PyImport_ImportModule("torch");
    PyObject* type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    PyErr_SetString(type ? type : PyExc_MemoryError, e.what_without_backtrace());
    Py_XDECREF(type);
    Py_XDECREF(torch);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// (q, k, positions, inv_freq, pair_axis, interleaved, inverse, q_out, k_out)
PyObject* py_rotary(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    const Tensor& q = tensor(a[0], "q");
    Maybe k = maybe(a[1], "k");
    const Call c(q);
    const attn_dtype dt = dtype_of(q);
    if (q.dim() != 3 || !head_dim(q.size(2))) bad("q must be [tokens, heads, d] with d 64, 128 or 160");
    const int64_t T = q.size(0), Hq = q.size(1), d = q.size(2), Hkv = k && k->dim() == 3 ? k->size(1) : 0;
    const auto type = q.scalar_type();
    const Rows x = rows16(c, q, "q", type, Hq, d, T);
    const Rows y = k ? rows16(c, *k, "k", type, Hkv, d, T) : Rows();
    const Rotary r = rotary(c, maybe(a[2], "positions"), maybe(a[3], "inv_freq"), maybe(a[4], "pair_axis"), d, T);
    if (!r.freq) bad("positions and inv_freq are needed");
    Maybe qo = maybe(a[7], "q_out"), ko = maybe(a[8], "k_out");
    if (ko && !k) bad("k_out without k");
    const Tensor nq = qo ? *qo : c.make({T, Hq, d}, type);
    const Tensor nk = !k ? Tensor() : (ko ? *ko : c.make({T, Hkv, d}, type));
    const Rows u = rows16(c, nq, "q_out", type, Hq, d, T);
    const Rows v = k ? rows16(c, nk, "k_out", type, Hkv, d, T) : Rows();
    if (T > 0)
      check(fn.rotary(dt, T, static_cast<int>(Hq), static_cast<int>(Hkv), static_cast<int>(d), x.p, x.ts, x.hs,
                      y.p, y.ts, y.hs, r.pos, r.axis_stride, r.axes, r.freq, r.axis, r.pairs, truth(a[5]),
                      truth(a[6]), u.p, u.ts, u.hs, v.p, v.ts, v.hs, c.stream()));
    return Py_BuildValue("(NN)", result(a[7], nq), k ? result(a[8], nk) : kept(Py_None));
  });
}

// (k, v, k_cache, v_cache, table, lens, cu_new, positions, inv_freq, pair_axis,
//  interleaved, key_pos, scores, lens_out, status)
PyObject* py_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 15, [&]() -> PyObject* {
    const Tensor& k = tensor(a[0], "k");
    const Tensor& v = tensor(a[1], "v");
    const Call c(k);
    const attn_dtype dt = dtype_of(k);
    if (k.dim() != 3 || !head_dim(k.size(2))) bad("k must be [tokens, heads, d] with d 64, 128 or 160");
    const int64_t T = k.size(0), H = k.size(1), d = k.size(2);
    const auto type = k.scalar_type();
    const Tensor &kc = tensor(a[2], "k_cache"), &vc = tensor(a[3], "v_cache"), &lens = tensor(a[5], "lens");
    const Pool kp = pool(c, kc, "k_cache", type), vp = pool(c, vc, "v_cache", type);
    if (kc.sizes() != vc.sizes() || kc.size(2) != H || kc.size(3) != d)
      bad("k_cache and v_cache must both be [num_pages, page_size, " + std::to_string(H) + ", " + std::to_string(d) + "]");
    const Tab t = table(c, tensor(a[4], "table"), lens, "table");
    const int64_t cap = t.width * kc.size(1);
    const Rows x = rows16(c, k, "k", type, H, d, T), y = rows16(c, v, "v", type, H, d, T);
    const Rotary r = rotary(c, maybe(a[7], "positions"), maybe(a[8], "inv_freq"), maybe(a[9], "pair_axis"), d, T);
    const auto pos = slots<int32_t>(c, maybe(a[11], "key_pos"), "key_pos", t.rows, H, cap);
    const auto sc = slots<float>(c, maybe(a[12], "scores"), "scores", t.rows, H, cap);
    Maybe lo = maybe(a[13], "lens_out");
    int32_t* lens_out = lo ? const_cast<int32_t*>(vec(c, *lo, "lens_out", t.rows)) : nullptr;
    if (lens_out && lens_out == t.lens) bad("lens_out must not be lens");
    check(fn.append(dt, static_cast<int>(t.rows), static_cast<int>(H), static_cast<int>(d), T, x.p, x.ts, x.hs,
                    y.p, y.ts, y.hs, kp.p, kp.ps, kp.ss, kp.hs, vp.p, vp.ps, vp.ss, vp.hs,
                    static_cast<int>(kc.size(0)), static_cast<int>(kc.size(1)), t.p, t.rs, t.width, t.lens,
                    vec(c, tensor(a[6], "cu_new"), "cu_new", t.rows + 1), r.pos, r.axis_stride, r.axes, r.freq,
                    r.axis, r.pairs, truth(a[10]), pos.p, pos.rs, pos.hs, sc.p, sc.rs, sc.hs, lens_out,
                    status_of(c, maybe(a[14], "status")), c.stream()));
    Py_RETURN_NONE;
  });
}

// What attention and the key weights share: (k_cache, table, lens, cu_q,
// alibi_slopes, prefix_table, prefix_lens, cu_prefix, q_pos, key_pos,
// prefix_key_pos, causal, window_left, window_right, softcap, scale) from a[0].
struct Read {
  attn_dtype dt;
  int B, P, Hq, Hkv, d;
  int64_t T, cap, pcap;
  at::ScalarType type;
  Rows q;
  Pool k;
  int pages, page;
  Tab own, prefix;
  const int32_t *cu_prefix = nullptr, *cu_q, *q_pos = nullptr;
  Slots<int32_t> pos, ppos;
  const float* slopes = nullptr;
  int64_t slopes_bs = 0;
  int causal, wl, wr;
  float cap_value, scale;
};
Read read_args(const Call& c, const Tensor& q, PyObject* const* a, bool bytes = false) {
  Read r;
  r.dt = dtype_of(q);
  r.type = q.scalar_type();
  if (q.dim() != 3 || !head_dim(q.size(2))) bad("q must be [tokens, heads, d] with d 64, 128 or 160");
  const Tensor& kc = tensor(a[0], "k_cache");
  r.k = pool(c, kc, "k_cache", bytes ? at::kFloat8_e4m3fn : r.type);
  r.T = q.size(0);
  const int64_t Hq = q.size(1), Hkv = kc.size(2), d = q.size(2);
  if (Hkv < 1 || Hq < 1 || Hq % Hkv || kc.size(3) != d || Hq > INT32_MAX)
    bad("q's " + std::to_string(Hq) + " heads of " + std::to_string(d) + " do not fit the cache's " +
        std::to_string(Hkv) + " heads of " + std::to_string(kc.size(3)));
  r.Hq = static_cast<int>(Hq);
  r.Hkv = static_cast<int>(Hkv);
  r.d = static_cast<int>(d);
  r.pages = static_cast<int>(kc.size(0));
  r.page = static_cast<int>(kc.size(1));
  r.q = rows16(c, q, "q", r.type, Hq, d, r.T);
  r.own = table(c, tensor(a[1], "table"), tensor(a[2], "lens"), "table");
  r.B = static_cast<int>(r.own.rows);
  r.cap = static_cast<int64_t>(r.own.width) * r.page;
  r.cu_q = vec(c, tensor(a[3], "cu_q"), "cu_q", r.own.rows + 1);
  if (Maybe s = maybe(a[4], "alibi_slopes")) {
    c.here(*s, "alibi_slopes");
    if (s->scalar_type() != at::kFloat || s->dim() != 2 || s->size(0) != r.B || s->size(1) != Hq ||
        (Hq > 1 && s->stride(1) != 1))
      bad("alibi_slopes must be fp32 [B, Hq] on the device, head stride 1");
    r.slopes = s->data_ptr<float>();
    r.slopes_bs = s->stride(0);
  }
  Maybe pt = maybe(a[5], "prefix_table"), pl = maybe(a[6], "prefix_lens"), pc = maybe(a[7], "cu_prefix");
  Maybe ppos = maybe(a[10], "prefix_key_pos");
  if ((pt != nullptr) != (pl != nullptr) || (pt != nullptr) != (pc != nullptr) || (ppos && !pt))
    bad("prefixes need prefix_table, prefix_lens and cu_prefix");
  r.P = pt ? static_cast<int>(pl->numel()) : 0;
  r.pcap = 0;
  if (r.P) {
    r.prefix = table(c, *pt, *pl, "prefix_table");
    r.cu_prefix = vec(c, *pc, "cu_prefix", r.P + 1);
    r.pcap = static_cast<int64_t>(r.prefix.width) * r.page;
  }
  if (Maybe t = maybe(a[8], "q_pos")) r.q_pos = vec(c, *t, "q_pos", r.T);
  Maybe pos = maybe(a[9], "key_pos");
  if ((pos || ppos) && !r.q_pos && r.T > 0) bad("key positions need q_pos");
  r.pos = slots<int32_t>(c, pos, "key_pos", r.B, Hkv, r.cap);
  if (r.P) r.ppos = slots<int32_t>(c, ppos, "prefix_key_pos", r.P, Hkv, r.pcap);
  r.causal = truth(a[11]);
  r.wl = small(a[12]);
  r.wr = small(a[13]);
  r.cap_value = static_cast<float>(real(a[14]));
  r.scale = static_cast<float>(real(a[15]));
  return r;
}

const float* lse_of(const Call& c, const Tensor& t, const Read& r) {
  c.here(t, "lse");
  if (t.scalar_type() != at::kFloat || t.dim() != 2 || t.size(0) != r.T || t.size(1) != r.Hq || !t.is_contiguous())
    bad("lse must be a dense fp32 CUDA tensor [tokens, heads]");
  return t.data_ptr<float>();
}

// (q, the 16 above, v_cache, out, lse, workspace, status)
PyObject* py_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 22, [&]() -> PyObject* {
    const Tensor& q = tensor(a[0], "q");
    const Call c(q);
    const Read r = read_args(c, q, a + 1);
    const Tensor& vc = tensor(a[17], "v_cache");
    const Pool v = pool(c, vc, "v_cache", r.type);
    if (vc.sizes() != tensor(a[1], "k_cache").sizes()) bad("k_cache and v_cache must have the same shape");
    Maybe go = maybe(a[18], "out"), gl = maybe(a[19], "lse");
    const Tensor out = go ? *go : c.make({r.T, r.Hq, r.d}, r.type);
    const Tensor lse = gl ? *gl : c.make({r.T, r.Hq}, at::kFloat);
    const Rows o = rows16(c, out, "out", r.type, r.Hq, r.d, r.T);
    const float* l = lse_of(c, lse, r);
    const Workspace w = workspace(c, maybe(a[20], "workspace"), fn.fwd_ws(r.B, r.P, r.Hq, r.Hkv, r.d, r.T));
    check(fn.fwd(r.dt, r.B, r.P, r.Hq, r.Hkv, r.d, r.T, r.q.p, r.q.ts, r.q.hs, r.k.p, r.k.ps, r.k.ss, r.k.hs, v.p,
                 v.ps, v.ss, v.hs, r.pages, r.page, r.own.p, r.own.rs, r.own.width, r.own.lens, r.prefix.p,
                 r.prefix.rs, r.prefix.width, r.prefix.lens, r.cu_prefix, r.cu_q, r.q_pos, r.pos.p, r.pos.rs,
                 r.pos.hs, r.ppos.p, r.ppos.rs, r.ppos.hs, r.slopes, r.slopes_bs, r.causal, r.wl, r.wr,
                 r.cap_value, r.scale, o.p, o.ts, o.hs, const_cast<float*>(l), w.p, w.bytes,
                 status_of(c, maybe(a[21], "status")), c.stream()));
    return Py_BuildValue("(NN)", result(a[18], out), result(a[19], lse));
  });
}

// (q, the 16 above, lse, scores, scores_out, prefix_scores, prefix_scores_out, workspace, status)
PyObject* py_weights(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 24, [&]() -> PyObject* {
    const Tensor& q = tensor(a[0], "q");
    const Call c(q);
    const Read r = read_args(c, q, a + 1);
    const float* lse = lse_of(c, tensor(a[17], "lse"), r);
    Maybe in = maybe(a[18], "scores"), pin = maybe(a[20], "prefix_scores");
    PyObject* oo = a[19] != Py_None ? a[19] : a[18];
    PyObject* po = a[21] != Py_None ? a[21] : a[20];
    Tensor fresh;
    Maybe out = maybe(oo, "scores_out"), pout = maybe(po, "prefix_scores_out");
    if (!out) {
      fresh = at::zeros({r.B, r.Hkv, r.cap}, at::TensorOptions().dtype(at::kFloat).device(c.device));
      out = &fresh;
    }
    if (pout && !r.P) bad("prefix_scores without prefixes");
    const auto si = slots<float>(c, in, "scores", r.B, r.Hkv, r.cap);
    const auto so = slots<float>(c, out, "scores_out", r.B, r.Hkv, r.cap);
    const auto pi = slots<float>(c, pin, "prefix_scores", r.P, r.Hkv, r.pcap);
    const auto ps = slots<float>(c, pout, "prefix_scores_out", r.P, r.Hkv, r.pcap);
    const Workspace w = workspace(c, maybe(a[22], "workspace"), fn.weights_ws());
    check(fn.weights(r.dt, r.B, r.P, r.Hq, r.Hkv, r.d, r.T, r.q.p, r.q.ts, r.q.hs, r.k.p, r.k.ps, r.k.ss, r.k.hs,
                     r.pages, r.page, r.own.p, r.own.rs, r.own.width, r.own.lens, r.prefix.p, r.prefix.rs,
                     r.prefix.width, r.prefix.lens, r.cu_prefix, r.cu_q, r.q_pos, r.pos.p, r.pos.rs, r.pos.hs,
                     r.ppos.p, r.ppos.rs, r.ppos.hs, r.slopes, r.slopes_bs, r.causal, r.wl, r.wr, r.cap_value,
                     r.scale, lse, si.p, si.rs, si.hs, so.p, so.rs, so.hs, pi.p, pi.rs, pi.hs, ps.p, ps.rs, ps.hs,
                     w.p, w.bytes, status_of(c, maybe(a[23], "status")), c.stream()));
    return Py_BuildValue("(NN)", result(oo, *out), kept(po));
  });
}

// (k_cache, v_cache, table, lens, scores, key_pos, next_pos, budget, recent,
//  scores_out, key_pos_out, lens_out, workspace, status)
PyObject* py_evict(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 14, [&]() -> PyObject* {
    const Tensor &kc = tensor(a[0], "k_cache"), &vc = tensor(a[1], "v_cache"), &lens = tensor(a[3], "lens");
    const Call c(kc);
    dtype_of(kc);
    const Pool k = pool(c, kc, "k_cache", kc.scalar_type()), v = pool(c, vc, "v_cache", kc.scalar_type());
    if (vc.sizes() != kc.sizes() || !head_dim(kc.size(3)))
      bad("k_cache and v_cache must have the same shape, with d 64, 128 or 160");
    const Tab t = table(c, tensor(a[2], "table"), lens, "table");
    const int64_t H = kc.size(2), cap = t.width * kc.size(1);
    PyObject* so = a[9] != Py_None ? a[9] : a[4];
    PyObject* po = a[10] != Py_None ? a[10] : a[5];
    PyObject* lo = a[11] != Py_None ? a[11] : a[3];
    const auto s = slots<float>(c, &tensor(a[4], "scores"), "scores", t.rows, H, cap);
    const auto p = slots<int32_t>(c, &tensor(a[5], "key_pos"), "key_pos", t.rows, H, cap);
    const auto s2 = slots<float>(c, &tensor(so, "scores_out"), "scores_out", t.rows, H, cap);
    const auto p2 = slots<int32_t>(c, &tensor(po, "key_pos_out"), "key_pos_out", t.rows, H, cap);
    int32_t* l2 = const_cast<int32_t*>(vec(c, tensor(lo, "lens_out"), "lens_out", t.rows));
    const int budget = small(a[7]), recent = small(a[8]);
    const Workspace w = workspace(c, maybe(a[12], "workspace"),
                                  fn.evict_ws(static_cast<int>(t.rows), static_cast<int>(H), t.width,
                                              static_cast<int>(kc.size(1)), budget));
    check(fn.evict(static_cast<int>(t.rows), static_cast<int>(H), static_cast<int>(kc.size(3)), k.p, k.ps, k.ss,
                   k.hs, v.p, v.ps, v.ss, v.hs, static_cast<int>(kc.size(0)), static_cast<int>(kc.size(1)), t.p,
                   t.rs, t.width, t.lens, s.p, s.rs, s.hs, p.p, p.rs, p.hs,
                   vec(c, tensor(a[6], "next_pos"), "next_pos", t.rows), budget, recent, s2.p, s2.rs, s2.hs, p2.p,
                   p2.rs, p2.hs, l2, w.p, w.bytes, status_of(c, maybe(a[13], "status")), c.stream()));
    return Py_BuildValue("(NNN)", kept(lo), kept(so), kept(po));
  });
}

const float* weight(const Call& c, Maybe t, const char* name, int64_t d) {
  if (!t) return nullptr;
  c.here(*t, name);
  if (t->scalar_type() != at::kFloat || t->dim() != 1 || t->size(0) != d || !t->is_contiguous())
    bad(std::string(name) + " must be a contiguous fp32 CUDA vector of " + std::to_string(d));
  return t->data_ptr<float>();
}

// (q, k, q_weight, k_weight, positions, inv_freq, pair_axis, interleaved, eps, q_out, k_out)
PyObject* py_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject* {
    const Tensor& q = tensor(a[0], "q");
    Maybe k = maybe(a[1], "k");
    const Call c(q);
    const attn_dtype dt = dtype_of(q);
    if (q.dim() != 3 || !head_dim(q.size(2))) bad("q must be [tokens, heads, d] with d 64, 128 or 160");
    const int64_t T = q.size(0), Hq = q.size(1), d = q.size(2), Hkv = k && k->dim() == 3 ? k->size(1) : 0;
    const auto type = q.scalar_type();
    const Rows x = rows16(c, q, "q", type, Hq, d, T);
    const Rows y = k ? rows16(c, *k, "k", type, Hkv, d, T) : Rows();
    const float *qw = weight(c, maybe(a[2], "q_weight"), "q_weight", d), *kw = weight(c, maybe(a[3], "k_weight"), "k_weight", d);
    const Rotary r = rotary(c, maybe(a[4], "positions"), maybe(a[5], "inv_freq"), maybe(a[6], "pair_axis"), d, T);
    Maybe qo = maybe(a[9], "q_out"), ko = maybe(a[10], "k_out");
    if (ko && !k) bad("k_out without k");
    const Tensor nq = qo ? *qo : c.make({T, Hq, d}, type);
    const Tensor nk = !k ? Tensor() : (ko ? *ko : c.make({T, Hkv, d}, type));
    const Rows u = rows16(c, nq, "q_out", type, Hq, d, T);
    const Rows v = k ? rows16(c, nk, "k_out", type, Hkv, d, T) : Rows();
    const int inter = truth(a[7]);
    const float eps = static_cast<float>(real(a[8]));
    if (T > 0)
      check(fn.norm(dt, T, static_cast<int>(Hq), static_cast<int>(Hkv), static_cast<int>(d), x.p, x.ts, x.hs, y.p,
                    y.ts, y.hs, qw, kw, eps, r.pos, r.axis_stride, r.axes, r.freq, r.axis, r.pairs, inter, u.p, u.ts,
                    u.hs, v.p, v.ts, v.hs, c.stream()));
    return Py_BuildValue("(NN)", result(a[9], nq), k ? result(a[10], nk) : kept(Py_None));
  });
}

// (dq_out, dk_out, q, k, q_weight, k_weight, positions, inv_freq, pair_axis, interleaved,
//  eps, dq, dk, dq_weight, dk_weight, workspace)
PyObject* py_norm_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 16, [&]() -> PyObject* {
    const Tensor& q = tensor(a[2], "q");
    Maybe k = maybe(a[3], "k"), dko = maybe(a[1], "dk_out");
    const Call c(q);
    const attn_dtype dt = dtype_of(q);
    if (q.dim() != 3 || !head_dim(q.size(2))) bad("q must be [tokens, heads, d] with d 64, 128 or 160");
    if ((k != nullptr) != (dko != nullptr)) bad("k and dk_out belong together");
    const int64_t T = q.size(0), Hq = q.size(1), d = q.size(2), Hkv = k && k->dim() == 3 ? k->size(1) : 0;
    const auto type = q.scalar_type();
    const Rows x = rows16(c, q, "q", type, Hq, d, T), dx = rows16(c, tensor(a[0], "dq_out"), "dq_out", type, Hq, d, T);
    const Rows y = k ? rows16(c, *k, "k", type, Hkv, d, T) : Rows();
    const Rows dy = k ? rows16(c, *dko, "dk_out", type, Hkv, d, T) : Rows();
    const float *qw = weight(c, maybe(a[4], "q_weight"), "q_weight", d), *kw = weight(c, maybe(a[5], "k_weight"), "k_weight", d);
    if (kw && !k) bad("k_weight without k");
    const Rotary r = rotary(c, maybe(a[6], "positions"), maybe(a[7], "inv_freq"), maybe(a[8], "pair_axis"), d, T);
    Maybe oq = maybe(a[11], "dq"), ok = maybe(a[12], "dk"), wq = maybe(a[13], "dq_weight"), wk = maybe(a[14], "dk_weight");
    if (ok && !k) bad("dk without k");
    if ((wq && !qw) || (wk && !kw)) bad("the gradient of a weight that the call does not have");
    const Tensor nq = oq ? *oq : c.make({T, Hq, d}, type);
    const Tensor nk = !k ? Tensor() : (ok ? *ok : c.make({T, Hkv, d}, type));
    const Tensor nwq = !qw ? Tensor() : (wq ? *wq : c.make({d}, at::kFloat));
    const Tensor nwk = !kw ? Tensor() : (wk ? *wk : c.make({d}, at::kFloat));
    const Rows u = rows16(c, nq, "dq", type, Hq, d, T);
    const Rows v = k ? rows16(c, nk, "dk", type, Hkv, d, T) : Rows();
    float* gq = const_cast<float*>(weight(c, qw ? &nwq : nullptr, "dq_weight", d));
    float* gk = const_cast<float*>(weight(c, kw ? &nwk : nullptr, "dk_weight", d));
    const int inter = truth(a[9]);
    const float eps = static_cast<float>(real(a[10]));
    const Workspace w = workspace(c, maybe(a[15], "workspace"),
                                  fn.norm_bwd_ws(T, static_cast<int>(Hq), static_cast<int>(Hkv), static_cast<int>(d)));
    check(fn.norm_bwd(dt, T, static_cast<int>(Hq), static_cast<int>(Hkv), static_cast<int>(d), dx.p, dx.ts, dx.hs, dy.p,
                      dy.ts, dy.hs, x.p, x.ts, x.hs, y.p, y.ts, y.hs, qw, kw, eps, r.pos, r.axis_stride, r.axes, r.freq,
                      r.axis, r.pairs, inter, u.p, u.ts, u.hs, v.p, v.ts, v.hs, gq, gk, w.p, w.bytes, c.stream()));
    return Py_BuildValue("(NNNN)", result(a[11], nq), k ? result(a[12], nk) : kept(Py_None),
                         qw ? result(a[13], nwq) : kept(Py_None), kw ? result(a[14], nwk) : kept(Py_None));
  });
}

struct BlockScales {  // [num_pages, page_size / block, Hkv]
  float* p;
  int64_t ps, bs, hs;
  int block;
};
BlockScales block_scales(const Call& c, const Tensor& t, const char* name, const Tensor& cache) {
  c.here(t, name);
  if (t.scalar_type() != at::kFloat || t.dim() != 3 || t.size(0) != cache.size(0) || t.size(1) < 1 ||
      cache.size(1) % t.size(1) || t.size(2) != cache.size(2))
    bad(std::string(name) + " must be fp32 [" + std::to_string(cache.size(0)) + ", page_size / block, " +
        std::to_string(cache.size(2)) + "] on the device");
  return {t.data_ptr<float>(), t.stride(0), t.stride(1), t.stride(2), static_cast<int>(cache.size(1) / t.size(1))};
}

// (k, v, k_cache, v_cache, k_scale, v_scale, table, lens, cu_new, positions, inv_freq,
//  pair_axis, interleaved, norm, k_weight, eps, key_pos, lens_out, status)
PyObject* py_append8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 19, [&]() -> PyObject* {
    const Tensor& k = tensor(a[0], "k");
    const Tensor& v = tensor(a[1], "v");
    const Call c(k);
    const attn_dtype dt = dtype_of(k);
    if (k.dim() != 3 || !head_dim(k.size(2))) bad("k must be [tokens, heads, d] with d 64, 128 or 160");
    const int64_t T = k.size(0), H = k.size(1), d = k.size(2);
    const auto type = k.scalar_type();
    const Tensor &kc = tensor(a[2], "k_cache"), &vc = tensor(a[3], "v_cache"), &lens = tensor(a[7], "lens");
    const Pool kp = pool(c, kc, "k_cache", at::kFloat8_e4m3fn), vp = pool(c, vc, "v_cache", at::kFloat8_e4m3fn);
    if (kc.sizes() != vc.sizes() || kc.size(2) != H || kc.size(3) != d)
      bad("k_cache and v_cache must both be [num_pages, page_size, " + std::to_string(H) + ", " + std::to_string(d) + "]");
    const BlockScales ks = block_scales(c, tensor(a[4], "k_scale"), "k_scale", kc);
    const BlockScales vs = block_scales(c, tensor(a[5], "v_scale"), "v_scale", vc);
    if (ks.block != vs.block) bad("k_scale and v_scale must have the same blocks");
    const Tab t = table(c, tensor(a[6], "table"), lens, "table");
    const int64_t cap = t.width * kc.size(1);
    const Rows x = rows16(c, k, "k", type, H, d, T), y = rows16(c, v, "v", type, H, d, T);
    const Rotary r = rotary(c, maybe(a[9], "positions"), maybe(a[10], "inv_freq"), maybe(a[11], "pair_axis"), d, T);
    const float* kw = weight(c, maybe(a[14], "k_weight"), "k_weight", d);
    const auto pos = slots<int32_t>(c, maybe(a[16], "key_pos"), "key_pos", t.rows, H, cap);
    Maybe lo = maybe(a[17], "lens_out");
    int32_t* lens_out = lo ? const_cast<int32_t*>(vec(c, *lo, "lens_out", t.rows)) : nullptr;
    if (lens_out && lens_out == t.lens) bad("lens_out must not be lens");
    const int inter = truth(a[12]), norm = a[13] == Py_None ? kw != nullptr : truth(a[13]);
    if (kw && !norm) bad("k_weight without the norm");
    check(fn.append8(dt, static_cast<int>(t.rows), static_cast<int>(H), static_cast<int>(d), T, x.p, x.ts, x.hs, y.p,
                     y.ts, y.hs, kp.p, kp.ps, kp.ss, kp.hs, vp.p, vp.ps, vp.ss, vp.hs, ks.p, ks.ps, ks.bs, ks.hs, vs.p,
                     vs.ps, vs.bs, vs.hs, static_cast<int>(kc.size(0)), static_cast<int>(kc.size(1)), ks.block, t.p,
                     t.rs, t.width, t.lens, vec(c, tensor(a[8], "cu_new"), "cu_new", t.rows + 1), r.pos, r.axis_stride,
                     r.axes, r.freq, r.axis, r.pairs, inter, norm, kw, static_cast<float>(real(a[15])), pos.p, pos.rs,
                     pos.hs, lens_out, status_of(c, maybe(a[18], "status")), c.stream()));
    Py_RETURN_NONE;
  });
}

// (q, the 16 of read_args, v_cache, k_scale, v_scale, out, lse, workspace, status)
PyObject* py_fwd8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 24, [&]() -> PyObject* {
    const Tensor& q = tensor(a[0], "q");
    const Call c(q);
    const Read r = read_args(c, q, a + 1, true);
    const Tensor &kc = tensor(a[1], "k_cache"), &vc = tensor(a[17], "v_cache");
    const Pool v = pool(c, vc, "v_cache", at::kFloat8_e4m3fn);
    if (vc.sizes() != kc.sizes()) bad("k_cache and v_cache must have the same shape");
    const BlockScales ks = block_scales(c, tensor(a[18], "k_scale"), "k_scale", kc);
    const BlockScales vs = block_scales(c, tensor(a[19], "v_scale"), "v_scale", vc);
    if (ks.block != vs.block) bad("k_scale and v_scale must have the same blocks");
    Maybe go = maybe(a[20], "out"), gl = maybe(a[21], "lse");
    const Tensor out = go ? *go : c.make({r.T, r.Hq, r.d}, r.type);
    const Tensor lse = gl ? *gl : c.make({r.T, r.Hq}, at::kFloat);
    const Rows o = rows16(c, out, "out", r.type, r.Hq, r.d, r.T);
    const float* l = lse_of(c, lse, r);
    const Workspace w = workspace(c, maybe(a[22], "workspace"), fn.fwd8_ws(r.B, r.P, r.Hq, r.Hkv, r.d, r.T));
    check(fn.fwd8(r.dt, r.B, r.P, r.Hq, r.Hkv, r.d, r.T, r.q.p, r.q.ts, r.q.hs, r.k.p, r.k.ps, r.k.ss, r.k.hs, v.p,
                  v.ps, v.ss, v.hs, ks.p, ks.ps, ks.bs, ks.hs, vs.p, vs.ps, vs.bs, vs.hs, r.pages, r.page, ks.block,
                  r.own.p, r.own.rs, r.own.width, r.own.lens, r.prefix.p, r.prefix.rs, r.prefix.width, r.prefix.lens,
                  r.cu_prefix, r.cu_q, r.q_pos, r.pos.p, r.pos.rs, r.pos.hs, r.ppos.p, r.ppos.rs, r.ppos.hs, r.slopes,
                  r.slopes_bs, r.causal, r.wl, r.wr, r.cap_value, r.scale, o.p, o.ts, o.hs, const_cast<float*>(l), w.p,
                  w.bytes, status_of(c, maybe(a[23], "status")), c.stream()));
    return Py_BuildValue("(NN)", result(a[20], out), result(a[21], lse));
  });
}

// A sequence of pools, each [num_pages, rows, heads, d] or [num_pages, rows, heads].
struct Pools {
  PyObject* seq;
  std::vector<attn_pool> pool;
  std::vector<const Tensor*> t;
  int64_t pages = -1, page_size = 0;
  explicit Pools(PyObject* o, const char* name) : seq(PySequence_Fast(o, "pools must be a list of tensors")) {
    if (!seq) throw Raised{};
    try {
      const Py_ssize_t n = PySequence_Fast_GET_SIZE(seq);
      for (Py_ssize_t i = 0; i < n; ++i) add(tensor(PySequence_Fast_GET_ITEM(seq, i), name), name);
    } catch (...) {
      Py_DECREF(seq);
      throw;
    }
  }
  ~Pools() { Py_DECREF(seq); }
  Pools(const Pools&) = delete;
  Pools& operator=(const Pools&) = delete;
  void add(const Tensor& x, const char* name) {
    const int64_t dims = x.dim(), e = static_cast<int64_t>(x.element_size());
    if ((dims != 4 && dims != 3) || (dims == 4 && x.size(3) > 1 && x.stride(3) != 1) || x.numel() == 0 || x.size(0) > INT32_MAX ||
        x.size(1) > 1024 || x.size(2) > INT32_MAX || (dims == 4 && x.size(3) * e > INT32_MAX))
      bad(std::string(name) + " must be tensors [num_pages, rows, heads, d] or [num_pages, rows, heads], not empty, "
          "at most 1024 rows a page, with a contiguous feature axis");
    if (pages >= 0 && x.size(0) != pages) bad(std::string(name) + " must have the same number of pages");
    pages = x.size(0);
    page_size = std::max(page_size, x.size(1));
    attn_pool p;
    p.base = x.data_ptr();
    p.rows = static_cast<int32_t>(x.size(1));
    if (dims == 4) {
      p.pieces = static_cast<int32_t>(x.size(2));
      p.bytes = static_cast<int32_t>(x.size(3) * e);
      p.piece_stride = used(x.stride(2), x.size(2), x.size(3)) * e;
    } else if (x.size(2) == 1 || x.stride(2) == 1) {
      p.pieces = 1;
      p.bytes = static_cast<int32_t>(x.size(2) * e);
      p.piece_stride = p.bytes;
    } else {
      p.pieces = static_cast<int32_t>(x.size(2));
      p.bytes = static_cast<int32_t>(e);
      p.piece_stride = x.stride(2) * e;
    }
    const int64_t row = static_cast<int64_t>(p.pieces) * p.bytes;
    p.row_stride = x.size(1) > 1 ? x.stride(1) * e : row;
    p.page_stride = x.size(0) > 1 ? x.stride(0) * e : row * p.rows;
    pool.push_back(p);
    t.push_back(&x);
  }
  void here(const Call& c, const char* name) const {
    for (const Tensor* x : t) c.here(*x, name);
  }
};
int page_size_of(PyObject* given, const Pools& p) {
  if (given != Py_None) return small(given);
  if (p.pool.empty()) bad("page_size is needed without pools");
  return static_cast<int>(p.page_size);
}
struct Cells {  // an int32 table [rows, width]
  int32_t* p = nullptr;
  int64_t rs = 0;
  int rows = 0, width = 1;
};
Cells cells(const Call& c, const Tensor& t, const char* name, int64_t rows, int64_t width) {
  c.here(t, name);
  if (t.scalar_type() != at::kInt || t.dim() != 2 || (rows >= 0 && t.size(0) != rows) || (width >= 0 && t.size(1) != width) ||
      t.size(1) < 1 || t.size(0) > INT32_MAX || t.size(1) > INT32_MAX || (t.size(1) > 1 && t.stride(1) != 1))
    bad(std::string(name) + " must be an int32 CUDA tensor [rows, width] with contiguous rows, of one shape with its output");
  return {t.data_ptr<int32_t>(), used(t.stride(0), t.size(0), t.size(1)), static_cast<int>(t.size(0)), static_cast<int>(t.size(1))};
}

// (pools, table, lens, held, refs, parents, room, table_out, lens_out, held_out, refs_out, page_size, workspace, status)
PyObject* py_fork(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 14, [&]() -> PyObject* {
    const Tensor &tab = tensor(a[1], "table"), &refs = tensor(a[4], "refs");
    const Call c(tab);
    const Pools pools(a[0], "pools");
    pools.here(c, "pools");
    const int64_t N = refs.numel();
    if (pools.pages >= 0 && N != pools.pages) bad("refs must have an entry for every page of the pools");
    const Cells t = cells(c, tab, "table", -1, -1);
    PyObject *to = a[7] != Py_None ? a[7] : a[1], *lo = a[8] != Py_None ? a[8] : a[2];
    PyObject *ho = a[9] != Py_None ? a[9] : a[3], *ro = a[10] != Py_None ? a[10] : a[4];
    const Cells u = cells(c, tensor(to, "table_out"), "table_out", t.rows, t.width);
    auto ints = [&](PyObject* o, const char* name, int64_t count) {
      return const_cast<int32_t*>(vec(c, tensor(o, name), name, count));
    };
    if (N > INT32_MAX) bad("refs has too many entries");
    const int32_t* room = a[6] == Py_None ? nullptr : ints(a[6], "room", t.rows);
    const Workspace w = workspace(c, maybe(a[12], "workspace"), fn.fork_ws(t.rows, t.width, static_cast<int>(N)));
    check(fn.fork(t.rows, static_cast<int>(N), page_size_of(a[11], pools), pools.pool.data(), static_cast<int>(pools.pool.size()),
                  t.p, t.rs, t.width, ints(a[2], "lens", t.rows), ints(a[3], "held", t.rows), ints(a[4], "refs", N),
                  ints(a[5], "parents", t.rows), room, u.p, u.rs, ints(lo, "lens_out", t.rows), ints(ho, "held_out", t.rows),
                  ints(ro, "refs_out", N), w.p, w.bytes, status_of(c, maybe(a[13], "status")), c.stream()));
    return Py_BuildValue("(NNNN)", kept(to), kept(lo), kept(ho), kept(ro));
  });
}

// (pools, table, held, refs, prefix_table, prefix_held, table_out, refs_out, prefix_table_out, live, page_size, workspace, status)
PyObject* py_compact(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&]() -> PyObject* {
    const Tensor &tab = tensor(a[1], "table"), &refs = tensor(a[3], "refs");
    const Call c(tab);
    const Pools pools(a[0], "pools");
    pools.here(c, "pools");
    const int64_t N = refs.numel();
    if (N > INT32_MAX || (pools.pages >= 0 && N != pools.pages)) bad("refs must have an entry for every page of the pools");
    auto ints = [&](PyObject* o, const char* name, int64_t count) {
      return const_cast<int32_t*>(vec(c, tensor(o, name), name, count));
    };
    PyObject *to = a[6] != Py_None ? a[6] : a[1], *ro = a[7] != Py_None ? a[7] : a[3], *po = a[8] != Py_None ? a[8] : a[4];
    const Cells t = cells(c, tab, "table", -1, -1), u = cells(c, tensor(to, "table_out"), "table_out", t.rows, t.width);
    Cells pt, pu;
    const int32_t* ph = nullptr;
    if (a[4] != Py_None) {
      pt = cells(c, tensor(a[4], "prefix_table"), "prefix_table", -1, -1);
      pu = cells(c, tensor(po, "prefix_table_out"), "prefix_table_out", pt.rows, pt.width);
      ph = ints(a[5], "prefix_held", pt.rows);
    } else if (a[5] != Py_None || a[8] != Py_None) {
      bad("prefix_held and prefix_table_out need prefix_table");
    }
    Maybe gl = maybe(a[9], "live");
    const Tensor live = gl ? *gl : c.make({1}, at::kInt);
    int32_t* lp = const_cast<int32_t*>(vec(c, live, "live", 1));
    const Workspace w = workspace(c, maybe(a[11], "workspace"), fn.compact_ws(static_cast<int>(N)));
    check(fn.compact(static_cast<int>(N), page_size_of(a[10], pools), pools.pool.data(), static_cast<int>(pools.pool.size()), t.rows,
                     t.p, t.rs, t.width, ints(a[2], "held", t.rows), u.p, u.rs, pt.rows, pt.p, pt.rs, pt.width, ph, pu.p, pu.rs,
                     ints(a[3], "refs", N), ints(ro, "refs_out", N), lp, w.p, w.bytes, status_of(c, maybe(a[12], "status")),
                     c.stream()));
    return Py_BuildValue("(NNNN)", result(a[9], live), kept(to), kept(ro), kept(po));
  });
}

// (src_pools, src_pages, dst_pages, dst_pools, page_size, status)
PyObject* py_copy(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 6, [&]() -> PyObject* {
    const Tensor& from = tensor(a[1], "src_pages");
    const Call c(from);
    const Pools src(a[0], "src_pools"), dst(a[3] != Py_None ? a[3] : a[0], "dst_pools");
    src.here(c, "src_pools");
    dst.here(c, "dst_pools");
    if (src.pool.size() != dst.pool.size()) bad("src_pools and dst_pools must have the same number of pools");
    const int64_t count = from.numel();
    if (count > INT32_MAX) bad("too many pages");
    const int32_t* f = vec(c, from, "src_pages", count);
    const int32_t* t = vec(c, tensor(a[2], "dst_pages"), "dst_pages", count);
    if (src.pool.empty()) Py_RETURN_NONE;
    for (size_t i = 0; i < src.t.size(); ++i)
      if (src.t[i]->scalar_type() != dst.t[i]->scalar_type() || src.t[i]->sizes().slice(1) != dst.t[i]->sizes().slice(1))
        bad("pools at the same place must have the same type and pages");
    std::vector<attn_pool> sp = src.pool, dp = dst.pool;
    for (size_t i = 0; i < sp.size(); ++i) {  // (rows of heads may be one run in one of them only)
      if (sp[i].pieces == dp[i].pieces) continue;
      attn_pool& one = sp[i].pieces == 1 ? sp[i] : dp[i];
      const attn_pool& many = sp[i].pieces == 1 ? dp[i] : sp[i];
      one.pieces = many.pieces;
      one.bytes = many.bytes;
      one.piece_stride = many.bytes;
    }
    check(fn.copy(static_cast<int>(count), f, t, static_cast<int>(src.pages), static_cast<int>(dst.pages),
                  page_size_of(a[4], src), sp.data(), dp.data(), static_cast<int>(sp.size()),
                  status_of(c, maybe(a[5], "status")), c.stream()));
    Py_RETURN_NONE;
  });
}

// bind(error class, addresses in the order of Fns)
PyObject* py_bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  constexpr Py_ssize_t count = sizeof(Fns) / sizeof(void*);
  if (n != 1 + count) {
    PyErr_SetString(PyExc_TypeError, "bind: wrong number of addresses");
    return nullptr;
  }
  void* at[count];
  for (Py_ssize_t i = 0; i < count; ++i) {
    at[i] = PyLong_AsVoidPtr(a[1 + i]);
    if (!at[i]) return PyErr_Occurred() ? nullptr : (PyErr_SetString(PyExc_ValueError, "bind: null address"), nullptr);
  }
  memcpy(&fn, at, sizeof fn);
  Py_XSETREF(attn_error, kept(a[0]));
  Py_RETURN_NONE;
}

#define METHOD(name, f) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD("bind", py_bind),       METHOD("rotary", py_rotary), METHOD("append", py_append),
                         METHOD("fwd", py_fwd),         METHOD("weights", py_weights), METHOD("evict", py_evict),
                         METHOD("norm", py_norm),       METHOD("norm_bwd", py_norm_bwd), METHOD("append8", py_append8),
                         METHOD("fwd8", py_fwd8),       METHOD("fork", py_fork),       METHOD("compact", py_compact),
                         METHOD("copy", py_copy),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&module); }
