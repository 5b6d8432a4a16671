// Native half of the Python entry points of the rotary, q/k norm, window,
// decode and paged calls: checks of the tensors, outputs and workspaces that were not
// given, and the call into the library, which is passed in as a table of its
// functions (so that the checked build is reached the same way).
//
// These operators run for a few microseconds on single tokens, where the same
// steps in Python around ctypes took several times as long as the kernel: call
// after call, q/k norms of 128 tokens took 20.2 us and take 6.0 (kernel 4.0), a
// decoded token of one sequence 16.9 and 8.2 (kernel 6.8).
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cstdint>
#include <optional>
#include <sstream>
#include <string>
#include <utility>
#include <vector>

#include "../../include/cpattn.h"

namespace {

// The library's functions, in the order of _CALLS in __init__.py.
struct Calls {
  decltype(&cpattn_rope_frequencies) rope_frequencies;
  decltype(&cpattn_rope_ex) rope_ex;
  decltype(&cpattn_qk_norm_rope) qk_norm_rope;
  decltype(&cpattn_qk_norm_rope_bwd_workspace_bytes) qk_norm_rope_bwd_bytes;
  decltype(&cpattn_qk_norm_rope_bwd) qk_norm_rope_bwd;
  decltype(&cpattn_fwd_window) fwd_window;
  decltype(&cpattn_bwd_window_workspace_bytes) bwd_window_bytes;
  decltype(&cpattn_bwd_window) bwd_window;
  decltype(&cpattn_fwd_window_varlen) fwd_window_varlen;
  decltype(&cpattn_bwd_window_varlen_workspace_bytes) bwd_window_varlen_bytes;
  decltype(&cpattn_bwd_window_varlen) bwd_window_varlen;
  decltype(&cpattn_decode_workspace_bytes) decode_bytes;
  decltype(&cpattn_decode) decode;
  decltype(&cpattn_append_paged) append_paged;
  decltype(&cpattn_decode_paged_workspace_bytes) decode_paged_bytes;
  decltype(&cpattn_decode_paged) decode_paged;
  decltype(&cpattn_decode_shared_workspace_bytes) decode_shared_bytes;
  decltype(&cpattn_decode_shared) decode_shared;
};

// ---------------------------------------------------------------- refusals
struct Refused {  // a Python exception to raise; type nullptr: one is set already
  PyObject* type;
  std::string what;
};
struct Failed {  // an error code of the library
  int rc;
};
template <class... T>
std::string text(const T&... parts) {
  std::ostringstream s;
  (s << ... << parts);
  return s.str();
}
[[noreturn]] void type_error(std::string what) { throw Refused{PyExc_TypeError, std::move(what)}; }
[[noreturn]] void value_error(std::string what) { throw Refused{PyExc_ValueError, std::move(what)}; }
void check(int rc) {
  if (rc != CPATTN_OK) throw Failed{rc};
}

std::string shape_text(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += text(i ? ", " : "", s[i]);
  return r + (s.size() == 1 ? ",)" : ")");
}
const char* type_text(at::ScalarType t) {
  return t == at::kBFloat16 ? "bfloat16" : t == at::kFloat ? "float32" : "int32";
}

// ---------------------------------------------------------------- arguments
// Reads a call's positional arguments one after another.
struct Args {
  PyObject* const* a;
  Py_ssize_t n, i = 0;
  PyObject* next() {
    if (i >= n) throw Refused{PyExc_SystemError, "too few arguments"};
    return a[i++];
  }
  PyObject* next_or_none() {  // nullptr for None
    PyObject* o = next();
    return o == Py_None ? nullptr : o;
  }
  int64_t integer(const char* name) { return integer_of(next(), name); }
  static int64_t integer_of(PyObject* o, const char* name) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused{nullptr, ""};
    if (v < INT_MIN || v > INT_MAX) value_error(text(name, " does not fit 32 bits"));
    return v;
  }
  // A count of keys: any that int32 cannot hold is all of them (and any
  // negative one -1, which the library refuses).
  int keys() {
    int over = 0;
    const long long v = PyLong_AsLongLongAndOverflow(next(), &over);
    if (v == -1 && !over && PyErr_Occurred()) throw Refused{nullptr, ""};
    return over > 0 || v > INT_MAX ? INT_MAX : over < 0 || v < 0 ? -1 : int(v);
  }
  double real() {
    const double v = PyFloat_AsDouble(next());
    if (v == -1.0 && PyErr_Occurred()) throw Refused{nullptr, ""};
    return v;
  }
  float scale() {  // None: the default
    if (i < n && a[i] == Py_None) {
      ++i;
      return 0.f;
    }
    return float(real());
  }
  const Calls& calls() {
    PyObject* o = next();
    if (!PyBytes_Check(o) || PyBytes_GET_SIZE(o) != sizeof(Calls))
      throw Refused{PyExc_SystemError, "not the library's function table"};
    return *reinterpret_cast<const Calls*>(PyBytes_AS_STRING(o));
  }
};

const at::Tensor& tensor(const char* name, PyObject* o, at::ScalarType type) {
  if (!THPVariable_Check(o) || THPVariable_Unpack(o).scalar_type() != type)
    type_error(text(name, " must be a ", type_text(type), " CUDA tensor"));
  return THPVariable_Unpack(o);
}

void same_shape(const char* name, const at::Tensor& t, at::IntArrayRef shape) {
  if (t.sizes() != shape) value_error(text(name, " has shape ", shape_text(t.sizes()), ", expected ", shape_text(shape)));
}

// Where a call runs: every tensor is on the current device; the stream given
// is current while the object lives, so that new tensors come from its memory
// and the caching allocator hands them to nobody else before it is done.
class Place {
 public:
  const at::Tensor& on(const at::Tensor& t) {
    if (!t.is_cuda()) type_error("every tensor must be a CUDA tensor");
    if (device_ < 0) device_ = c10::cuda::current_device();
    const int at = t.get_device();
    if (at != device_)
      value_error(text("a tensor is on cuda:", at, " but the current CUDA device is cuda:", device_,
                       "; call under torch.cuda.device(cuda:", at, ")"));
    return t;
  }
  void stream(PyObject* s) {  // torch.cuda.Stream, or nullptr; after the tensors
    if (s) {
      const int64_t id = field(s, "stream_id"), index = field(s, "device_index"), type = field(s, "device_type");
      if (index != device_)
        value_error(text("the stream belongs to cuda:", index, ", the current CUDA device is cuda:", device_));
      guard_.emplace(c10::cuda::CUDAStream::unpack3(id, c10::DeviceIndex(index), c10::DeviceType(type)));
    }
    stream_ = c10::cuda::getCurrentCUDAStream(c10::DeviceIndex(device_)).stream();
  }
  void* handle() const { return stream_; }
  at::Tensor empty(at::IntArrayRef shape, at::ScalarType type) const {
    return at::detail::empty_cuda(shape, type, at::Device(at::kCUDA, c10::DeviceIndex(device_)), std::nullopt);
  }

 private:
  static int64_t field(PyObject* s, const char* name) {
    PyObject* v = PyObject_GetAttrString(s, name);
    if (!v) throw Refused{nullptr, ""};
    const long long r = PyLong_AsLongLong(v);
    Py_DECREF(v);
    if (r == -1 && PyErr_Occurred()) throw Refused{nullptr, ""};
    return r;
  }
  int device_ = -1;
  cudaStream_t stream_ = nullptr;
  std::optional<c10::cuda::CUDAStreamGuard> guard_;
};

// A contiguous tensor of a type and, where given, a shape.
const at::Tensor& dense(const char* name, PyObject* o, at::ScalarType type, Place& place) {
  const at::Tensor& t = tensor(name, o, type);
  if (!t.is_contiguous()) value_error(text(name, " must be contiguous"));
  return place.on(t);
}
const at::Tensor& dense(const char* name, PyObject* o, at::ScalarType type, at::IntArrayRef shape, Place& place) {
  same_shape(name, tensor(name, o, type), shape);
  return dense(name, o, type, place);
}

// The library's sizes are ints.
void sizes_fit(const at::Tensor& t) {
  for (const int64_t s : t.sizes())
    if (s > INT_MAX) check(CPATTN_ERR_INVALID_ARG);
}

// cpattn_rows of a bf16 tensor [b, n, h, d] with contiguous heads. A stride of
// a dimension of one element means nothing and is not passed on.
cpattn_rows rows_of(const char* name, const at::Tensor& t) {
  if (t.dim() != 4) value_error(text(name, " must be [b, n, h, d]"));
  sizes_fit(t);
  const auto size = t.sizes(), stride = t.strides();
  if (stride[3] != 1 || (size[2] > 1 && stride[2] != size[3]))
    value_error(text(name, " must have contiguous heads and features"));
  return {t.data_ptr(), size[0] > 1 ? stride[0] : 0, size[1] > 1 ? stride[1] : size[2] * size[3]};
}
cpattn_rows rows(const char* name, PyObject* o, Place& place) {
  return rows_of(name, place.on(tensor(name, o, at::kBFloat16)));
}
cpattn_rows rows(const char* name, PyObject* o, at::IntArrayRef shape, Place& place) {
  same_shape(name, tensor(name, o, at::kBFloat16), shape);
  return rows(name, o, place);
}

// An output, given or (once the call is known to be made) new.
struct Out {
  PyObject* given;
  at::Tensor made;
  cpattn_rows at{nullptr, 0, 0};
  void* data() const { return at.data; }
  // the Python object for the caller
  PyObject* take() {
    if (!given) return THPVariable_Wrap(std::move(made));
    Py_INCREF(given);
    return given;
  }
};
Out out_dense(const char* name, PyObject* o, at::IntArrayRef shape, at::ScalarType type, Place& place) {
  Out r{o, {}};
  if (o) r.at.data = dense(name, o, type, shape, place).data_ptr();
  return r;
}
Out out_rows(const char* name, PyObject* o, at::IntArrayRef shape, Place& place) {
  Out r{o, {}};
  if (o) r.at = rows(name, o, shape, place);
  return r;
}
void make(Out& r, at::IntArrayRef shape, at::ScalarType type, const Place& place) {
  if (r.given) return;
  r.made = place.empty(shape, type);
  r.at.data = r.made.data_ptr();
  if (shape.size() == 4) r.at = {r.at.data, shape[1] * shape[2] * shape[3], shape[2] * shape[3]};
}

// The workspace given, or a new one of `need` bytes (none when need is 0).
struct Workspace {
  at::Tensor made;
  void* data = nullptr;
  size_t bytes = 0;
  void given(PyObject* o, Place& place) {
    if (!THPVariable_Check(o)) type_error("workspace must be a CUDA tensor");
    const at::Tensor& t = place.on(THPVariable_Unpack(o));
    if (!t.is_contiguous()) value_error("workspace must be a contiguous CUDA tensor");
    data = t.data_ptr();
    bytes = size_t(t.numel()) * t.element_size();
  }
  void make(size_t need, const Place& place) {
    if (need == 0) return;
    bytes = need;
    made = place.empty({int64_t(need)}, at::kByte);
    data = made.data_ptr();
  }
};

PyObject* results(std::initializer_list<Out*> outs) {
  PyObject* r = PyTuple_New(Py_ssize_t(outs.size()));
  if (!r) throw Refused{nullptr, ""};
  Py_ssize_t i = 0;
  for (Out* o : outs) {
    PyObject* t = o->take();
    if (!t) {
      Py_DECREF(r);
      throw Refused{nullptr, ""};
    }
    PyTuple_SET_ITEM(r, i++, t);
  }
  return r;
}

// The library's call, without the interpreter's lock (a launch may wait for
// room in the stream's queue).
template <class F>
void launch(F f) {
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = f();
  Py_END_ALLOW_THREADS
  check(rc);
}

// ---------------------------------------------------------------- rotation plan
// Arguments base, cp, rank, s, cu_seqlens, positions, layout, rot_dim,
// inv_freq, magnitude for b x n tokens of heads of d features.
struct Plan {
  cpattn_rotary r{};
  std::vector<double> freq;  // formed here when none were given
};
void read_plan(Plan& p, Args& a, const Calls& calls, int64_t b, int64_t n, int64_t d, Place& place) {
  const double base = a.real();
  const int64_t cp = a.integer("cp");
  PyObject* rank = a.next_or_none();
  PyObject* s = a.next_or_none();
  PyObject* cu = a.next_or_none();
  PyObject* pos = a.next_or_none();
  PyObject* layout = a.next_or_none();
  PyObject* rot_dim = a.next_or_none();
  PyObject* inv_freq = a.next_or_none();
  if (!layout) value_error("layout must be one of ['half', 'interleaved']");
  p.r.layout = int(Args::integer_of(layout, "layout"));
  int64_t rot = rot_dim ? Args::integer_of(rot_dim, "rot_dim") : d;
  if (inv_freq) {
    if (!THPVariable_Check(inv_freq)) type_error("inv_freq must be a contiguous fp64 host vector");
    const at::Tensor& f = THPVariable_Unpack(inv_freq);
    if (f.scalar_type() != at::kDouble || !f.is_cpu() || f.dim() != 1 || !f.is_contiguous())
      type_error("inv_freq must be a contiguous fp64 host vector");
    const int64_t pairs = f.size(0);
    if (rot_dim && 2 * pairs != rot)
      value_error(text("inv_freq has ", pairs, " values, rot_dim ", rot, " needs ", rot / 2));
    rot = 2 * pairs < INT_MAX ? 2 * pairs : INT_MAX;
    p.r.inv_freq = f.const_data_ptr<double>();
  } else {
    if (rot < 2 || rot > d) check(CPATTN_ERR_INVALID_ARG);
    p.freq.resize(size_t(rot / 2));
    check(calls.rope_frequencies(int(rot), base, CPATTN_ROPE_UNSCALED, 1.0, 0.0, 1.0, 32.0, p.freq.data()));
    p.r.inv_freq = p.freq.data();
  }
  p.r.rot_dim = int(rot);
  p.r.magnitude = float(a.real());
  p.r.cp = int(cp);
  p.r.rank = rank ? int(Args::integer_of(rank, "rank")) : -1;
  const int64_t len = s ? Args::integer_of(s, "s") : rank ? n * cp : n;
  if (len < INT_MIN || len > INT_MAX) value_error("s does not fit 32 bits");
  p.r.s = int(len);
  if (cu) {
    if (!THPVariable_Check(cu) || THPVariable_Unpack(cu).scalar_type() != at::kInt ||
        !THPVariable_Unpack(cu).is_contiguous())
      type_error("cu_seqlens must be a contiguous int32 CUDA tensor");
    const at::Tensor& t = place.on(THPVariable_Unpack(cu));
    if (t.numel() < 2 || t.numel() > INT_MAX) value_error("cu_seqlens must hold nseq + 1 offsets, nseq >= 1");
    p.r.cu_seqlens = t.const_data_ptr<int>();
    p.r.nseq = int(t.numel() - 1);
  }
  if (pos) {
    const at::Tensor& t = place.on(tensor("positions", pos, at::kInt));
    if (t.sizes() != at::IntArrayRef({n}) && t.sizes() != at::IntArrayRef({b, n}))
      value_error(text("positions has shape ", shape_text(t.sizes()), ", expected (", n, ",) or (", b, ", ", n, ")"));
    if (n > 1 && t.stride(-1) != 1) value_error("the positions of a sequence must be contiguous");
    p.r.positions = t.const_data_ptr<int>();
    p.r.positions_batch = t.dim() == 2 && b > 1 ? t.stride(0) : 0;
  }
}

// ---------------------------------------------------------------- the calls
PyObject* rope(Args& a) {
  const Calls& calls = a.calls();
  Place place;
  PyObject* xo = a.next();
  PyObject* outo = a.next();
  const cpattn_rows x = rows("x", xo, place);
  const auto size = THPVariable_Unpack(xo).sizes();
  const cpattn_rows y = outo == xo ? x : rows("out", outo, size, place);
  Plan plan;
  read_plan(plan, a, calls, size[0], size[1], size[3], place);
  const int inverse = int(a.integer("inverse"));
  place.stream(a.next_or_none());
  launch([&] {
    return calls.rope_ex(&x, &y, int(size[0]), int(size[1]), int(size[2]), int(size[3]), &plan.r, inverse,
                         place.handle());
  });
  Py_INCREF(outo);
  return outo;
}

// q, k and their weights.
struct NormInputs {
  cpattn_rows q, k;
  const void* wq;
  const void* wk;
  int fp32, b, n, hq, hkv, d;
  at::IntArrayRef q_size, k_size;
};
NormInputs read_norm(Args& a, Place& place) {
  NormInputs r;
  PyObject* q = a.next();
  PyObject* k = a.next();
  PyObject* wq = a.next();
  PyObject* wk = a.next();
  r.q = rows("q", q, place);
  r.k = rows("k", k, place);
  r.q_size = THPVariable_Unpack(q).sizes();
  r.k_size = THPVariable_Unpack(k).sizes();
  if (r.k_size[0] != r.q_size[0] || r.k_size[1] != r.q_size[1] || r.k_size[3] != r.q_size[3])
    value_error("k must be [b, n, hkv, d] matching q");
  if (!THPVariable_Check(wq)) type_error("q_weight and k_weight must be bf16 or fp32 CUDA tensors");
  const at::ScalarType type = THPVariable_Unpack(wq).scalar_type();
  if (type != at::kFloat && type != at::kBFloat16) type_error("q_weight and k_weight must be bf16 or fp32 CUDA tensors");
  r.b = int(r.q_size[0]);
  r.n = int(r.q_size[1]);
  r.hq = int(r.q_size[2]);
  r.hkv = int(r.k_size[2]);
  r.d = int(r.q_size[3]);
  r.wq = dense("q_weight", wq, type, {r.d}, place).data_ptr();
  r.wk = dense("k_weight", wk, type, {r.d}, place).data_ptr();
  r.fp32 = type == at::kFloat;
  return r;
}

PyObject* qk_norm_rope(Args& a) {
  const Calls& calls = a.calls();
  Place place;
  const NormInputs in = read_norm(a, place);
  const float eps = float(a.real());
  Plan plan;
  read_plan(plan, a, calls, in.b, in.n, in.d, place);
  Out q = out_rows("q_out", a.next_or_none(), in.q_size, place), k = out_rows("k_out", a.next_or_none(), in.k_size, place);
  place.stream(a.next_or_none());
  make(q, in.q_size, at::kBFloat16, place);
  make(k, in.k_size, at::kBFloat16, place);
  launch([&] {
    return calls.qk_norm_rope(&in.q, &in.k, in.wq, in.wk, in.fp32, eps, &q.at, &k.at, in.b, in.n, in.hq, in.hkv, in.d,
                              &plan.r, place.handle());
  });
  return results({&q, &k});
}

PyObject* qk_norm_rope_bwd(Args& a) {
  const Calls& calls = a.calls();
  Place place;
  const NormInputs in = read_norm(a, place);
  const cpattn_rows gq = rows("dq_out", a.next(), in.q_size, place), gk = rows("dk_out", a.next(), in.k_size, place);
  const float eps = float(a.real());
  Plan plan;
  read_plan(plan, a, calls, in.b, in.n, in.d, place);
  Out q = out_rows("dq", a.next_or_none(), in.q_size, place), k = out_rows("dk", a.next_or_none(), in.k_size, place);
  Out wq = out_dense("dq_weight", a.next_or_none(), {in.d}, at::kFloat, place);
  Out wk = out_dense("dk_weight", a.next_or_none(), {in.d}, at::kFloat, place);
  Workspace ws;
  PyObject* given = a.next_or_none();
  if (given) ws.given(given, place);
  place.stream(a.next_or_none());
  make(q, in.q_size, at::kBFloat16, place);
  make(k, in.k_size, at::kBFloat16, place);
  make(wq, {in.d}, at::kFloat, place);
  make(wk, {in.d}, at::kFloat, place);
  if (!given) ws.make(calls.qk_norm_rope_bwd_bytes(in.d), place);
  launch([&] {
    return calls.qk_norm_rope_bwd(&in.q, &in.k, in.wq, in.wk, in.fp32, eps, &gq, &gk, &q.at, &k.at,
                                  static_cast<float*>(wq.data()), static_cast<float*>(wk.data()), ws.data, ws.bytes,
                                  in.b, in.n, in.hq, in.hkv, in.d, &plan.r, place.handle());
  });
  return results({&q, &k, &wq, &wk});
}

// q [b, sq, hq, d] and k, v [b, skv, hkv, d]; packed: without b.
struct AttnInputs {
  const void* q;
  const void* k;
  const void* v;
  at::IntArrayRef q_size, k_size;
  int b, sq, skv, hq, hkv, d;
  std::vector<int64_t> lse_size;
};
AttnInputs read_attn(Args& a, bool packed, Place& place) {
  AttnInputs r;
  PyObject* q = a.next();
  PyObject* k = a.next();
  PyObject* v = a.next();
  const char* want = packed ? "packed q must be [total, hq, d] and k, v [total, hkv, d]"
                            : "q must be [b, sq, hq, d] and k, v [b, skv, hkv, d]";
  const size_t dims = packed ? 3 : 4;
  r.q_size = tensor("q", q, at::kBFloat16).sizes();
  r.k_size = tensor("k", k, at::kBFloat16).sizes();
  if (r.q_size.size() != dims || r.k_size.size() != dims || r.k_size[0] != r.q_size[0] || r.k_size.back() != r.q_size.back())
    value_error(want);
  sizes_fit(THPVariable_Unpack(q));
  sizes_fit(THPVariable_Unpack(k));
  r.q = dense("q", q, at::kBFloat16, place).data_ptr();
  r.k = dense("k", k, at::kBFloat16, place).data_ptr();
  r.v = dense("v", v, at::kBFloat16, r.k_size, place).data_ptr();
  r.b = packed ? 1 : int(r.q_size[0]);
  r.sq = int(r.q_size[dims - 3]);
  r.skv = int(r.k_size[dims - 3]);
  r.hq = int(r.q_size[dims - 2]);
  r.hkv = int(r.k_size[dims - 2]);
  r.d = int(r.q_size[dims - 1]);
  if (packed)
    r.lse_size = {r.hq, r.sq};
  else
    r.lse_size = {r.b, r.hq, r.sq};
  return r;
}

// Sample offsets: an int32 buffer of the host, held while the object lives.
class Offsets {
 public:
  Offsets() = default;
  ~Offsets() {
    if (view_.obj) PyBuffer_Release(&view_);
  }
  Offsets(const Offsets&) = delete;
  Offsets& operator=(const Offsets&) = delete;
  void read(PyObject* o, int64_t total) {
    if (PyObject_GetBuffer(o, &view_, PyBUF_SIMPLE) != 0) throw Refused{nullptr, ""};
    const int64_t n = view_.len / int64_t(sizeof(int));
    if (n < 1 || n > INT_MAX || data()[n - 1] != total) value_error("cu_seqlens must end at the packed length");
    nseq = int(n - 1);
  }
  const int* data() const { return static_cast<const int*>(view_.buf); }
  int nseq = 0;

 private:
  Py_buffer view_{};
};

PyObject* fwd_window_any(Args& a, bool packed) {
  const Calls& calls = a.calls();
  Place place;
  const AttnInputs in = read_attn(a, packed, place);
  Offsets cu;
  if (packed) cu.read(a.next(), in.sq);
  const int window = a.keys(), sinks = a.keys();
  const float scale = a.scale();
  Out o = out_dense("o", a.next_or_none(), in.q_size, at::kBFloat16, place);
  Out lse = out_dense("lse", a.next_or_none(), in.lse_size, at::kFloat, place);
  place.stream(a.next_or_none());
  make(o, in.q_size, at::kBFloat16, place);
  make(lse, in.lse_size, at::kFloat, place);
  launch([&] {
    float* l = static_cast<float*>(lse.data());
    if (packed)
      return calls.fwd_window_varlen(in.q, in.k, in.v, o.data(), l, cu.data(), cu.nseq, in.hq, in.hkv, in.d, window,
                                     sinks, scale, place.handle());
    return calls.fwd_window(in.q, in.k, in.v, o.data(), l, in.b, in.sq, in.skv, in.hq, in.hkv, in.d, window, sinks,
                            scale, place.handle());
  });
  return results({&o, &lse});
}
PyObject* fwd_window(Args& a) { return fwd_window_any(a, false); }
PyObject* fwd_window_varlen(Args& a) { return fwd_window_any(a, true); }

PyObject* bwd_window_any(Args& a, bool packed) {
  const Calls& calls = a.calls();
  Place place;
  const AttnInputs in = read_attn(a, packed, place);
  const void* o = dense("o", a.next(), at::kBFloat16, in.q_size, place).data_ptr();
  const float* lse = static_cast<const float*>(dense("lse", a.next(), at::kFloat, in.lse_size, place).data_ptr());
  const void* grad = dense("do", a.next(), at::kBFloat16, in.q_size, place).data_ptr();
  Offsets cu;
  if (packed) cu.read(a.next(), in.sq);
  const int window = a.keys(), sinks = a.keys();
  const float scale = a.scale();
  Out dq = out_dense("dq", a.next_or_none(), in.q_size, at::kBFloat16, place);
  Out dk = out_dense("dk", a.next_or_none(), in.k_size, at::kBFloat16, place);
  Out dv = out_dense("dv", a.next_or_none(), in.k_size, at::kBFloat16, place);
  Workspace ws;
  PyObject* given = a.next_or_none();
  if (given) ws.given(given, place);
  place.stream(a.next_or_none());
  make(dq, in.q_size, at::kBFloat16, place);
  make(dk, in.k_size, at::kBFloat16, place);
  make(dv, in.k_size, at::kBFloat16, place);
  if (!given) {
    // a shape that the call refuses needs none
    const size_t need = packed ? calls.bwd_window_varlen_bytes(cu.data(), cu.nseq, in.hq, in.hkv, in.d, window, sinks)
                               : calls.bwd_window_bytes(in.b, in.sq, in.skv, in.hq, in.hkv, in.d, window, sinks);
    ws.make(need > 0 ? need : 16, place);
  }
  launch([&] {
    if (packed)
      return calls.bwd_window_varlen(in.q, in.k, in.v, o, lse, grad, dq.data(), dk.data(), dv.data(), ws.data, ws.bytes,
                                     cu.data(), cu.nseq, in.hq, in.hkv, in.d, window, sinks, scale, place.handle());
    return calls.bwd_window(in.q, in.k, in.v, o, lse, grad, dq.data(), dk.data(), dv.data(), ws.data, ws.bytes, in.b,
                            in.sq, in.skv, in.hq, in.hkv, in.d, window, sinks, scale, place.handle());
  });
  return results({&dq, &dk, &dv});
}
PyObject* bwd_window(Args& a) { return bwd_window_any(a, false); }
PyObject* bwd_window_varlen(Args& a) { return bwd_window_any(a, true); }

// A stride of a dimension of one element means nothing.
int64_t used(int64_t size, int64_t stride) { return size > 1 ? stride : 0; }

PyObject* decode(Args& a) {
  const Calls& calls = a.calls();
  Place place;
  const at::Tensor& q = place.on(tensor("q", a.next(), at::kBFloat16));
  const at::Tensor& k = place.on(tensor("k_cache", a.next(), at::kBFloat16));
  const at::Tensor& v = place.on(tensor("v_cache", a.next(), at::kBFloat16));
  if (q.dim() != 3 || k.dim() != 4) value_error("q must be [b, hq, d] and k_cache, v_cache [b, cap, hkv, d]");
  const int64_t b = q.size(0), hq = q.size(1), d = q.size(2), cap = k.size(1), hkv = k.size(2);
  if (k.size(0) != b || k.size(3) != d || v.sizes() != k.sizes())
    value_error("k_cache and v_cache must be [b, cap, hkv, d] matching q");
  const auto qs = q.strides(), ks = k.strides(), vs = v.strides();
  if (qs[2] != 1 || ks[3] != 1 || vs[3] != 1 || (hq > 1 && qs[1] != d))
    value_error("q's heads and the features of q and of the cache must be contiguous");
  sizes_fit(q);
  sizes_fit(k);
  const void* lengths = dense("lengths", a.next(), at::kInt, {b}, place).data_ptr();
  const int window = a.keys(), sinks = a.keys();
  const float scale = a.scale();
  Out o = out_dense("o", a.next_or_none(), q.sizes(), at::kBFloat16, place);
  Out lse = out_dense("lse", a.next_or_none(), {b, hq}, at::kFloat, place);
  Workspace ws;
  PyObject* given = a.next_or_none();
  if (given) ws.given(given, place);
  place.stream(a.next_or_none());
  make(o, q.sizes(), at::kBFloat16, place);
  make(lse, {b, hq}, at::kFloat, place);
  if (!given) ws.make(calls.decode_bytes(int(b), int(hq), int(hkv), int(d), int(cap), window, sinks), place);
  launch([&] {
    return calls.decode(q.data_ptr(), k.data_ptr(), v.data_ptr(), static_cast<const int*>(lengths), o.data(),
                        static_cast<float*>(lse.data()), ws.data, ws.bytes, int(b), int(hq), int(hkv), int(d), int(cap),
                        used(b, qs[0]), used(b, ks[0]), used(cap, ks[1]), used(hkv, ks[2]), used(b, vs[0]),
                        used(cap, vs[1]), used(hkv, vs[2]), window, sinks, scale, place.handle());
  });
  return results({&o, &lse});
}

// Arguments k_pages, v_pages, tables: a cache in pages of heads of d features
// (cpattn_pages), with its KV heads and the tables' rows.
struct Pages {
  cpattn_pages p{};
  int64_t hkv = 0, rows = 0, cap = 0;
};
Pages read_pages(Args& a, int64_t d, Place& place) {
  Pages r;
  const at::Tensor& k = place.on(tensor("k_pages", a.next(), at::kBFloat16));
  const at::Tensor& v = place.on(tensor("v_pages", a.next(), at::kBFloat16));
  const at::Tensor& t = place.on(tensor("tables", a.next(), at::kInt));
  if (k.dim() != 4 || k.size(3) != d || v.sizes() != k.sizes())
    value_error(text("k_pages and v_pages must be [pages, page_size, hkv, ", d, "]"));
  const auto ks = k.strides(), vs = v.strides();
  if (ks[3] != 1 || vs[3] != 1) value_error("the features of the pages must be contiguous");
  if (t.dim() != 2 || (t.size(1) > 1 && t.stride(1) != 1))
    value_error("tables must be [sequences, columns] with contiguous rows");
  sizes_fit(k);
  sizes_fit(t);
  r.hkv = k.size(2);
  r.rows = t.size(0);
  r.cap = t.size(1) * k.size(1);
  r.p.k = k.data_ptr();
  r.p.v = v.data_ptr();
  r.p.pages = int(k.size(0));
  r.p.page_size = int(k.size(1));
  r.p.table_cols = int(t.size(1));
  r.p.tables = t.const_data_ptr<int>();
  r.p.tables_row = used(t.size(0), t.stride(0));
  r.p.k_page = used(k.size(0), ks[0]);
  r.p.k_token = ks[1];
  r.p.k_head = used(k.size(2), ks[2]);
  r.p.v_page = used(k.size(0), vs[0]);
  r.p.v_token = vs[1];
  r.p.v_head = used(k.size(2), vs[2]);
  return r;
}

PyObject* append_paged(Args& a) {
  const Calls& calls = a.calls();
  Place place;
  PyObject* ko = a.next();
  PyObject* vo = a.next();
  const cpattn_rows k = rows("k", ko, place);
  const auto size = THPVariable_Unpack(ko).sizes();
  const cpattn_rows v = rows("v", vo, size, place);
  const int64_t b = size[0], n = size[1], hkv = size[2], d = size[3];
  const Pages pages = read_pages(a, d, place);
  if (pages.hkv != hkv) value_error(text("the pages hold ", pages.hkv, " KV heads, k has ", hkv));
  PyObject* lo = a.next();
  PyObject* cuo = a.next_or_none();
  int64_t seqs = b;
  const int* cu = nullptr;
  if (cuo) {
    const at::Tensor& t = dense("cu_tokens", cuo, at::kInt, place);
    if (t.dim() != 1 || t.size(0) < 2 || t.size(0) > INT_MAX) value_error("cu_tokens must hold seqs + 1 offsets, seqs >= 1");
    if (b != 1) value_error("with cu_tokens, k and v must be [1, n, hkv, d]");
    cu = t.const_data_ptr<int>();
    seqs = t.size(0) - 1;
  }
  const int* lengths = static_cast<const int*>(dense("lengths", lo, at::kInt, {seqs}, place).data_ptr());
  if (pages.rows != seqs) value_error(text("tables has ", pages.rows, " rows for ", seqs, " sequences"));
  PyObject* qo = a.next_or_none();
  cpattn_rows q{nullptr, 0, 0};
  std::vector<int64_t> q_size;
  if (qo) {
    q = rows("q", qo, place);
    q_size = THPVariable_Unpack(qo).sizes().vec();
    if (q_size[0] != b || q_size[1] != n || q_size[3] != d) value_error("q must be [b, n, hq, d] matching k");
  }
  const bool rotate = a.integer("rotate") != 0;
  Plan plan;
  read_plan(plan, a, calls, b, n, d, place);
  PyObject* outo = a.next_or_none();
  if (outo && !qo) value_error("q_out goes with q");
  Out out = out_rows("q_out", outo, q_size, place);
  place.stream(a.next_or_none());
  if (qo) make(out, q_size, at::kBFloat16, place);
  launch([&] {
    return calls.append_paged(&k, &v, &pages.p, lengths, cu, int(seqs), qo ? &q : nullptr, qo ? &out.at : nullptr, int(b),
                              int(n), qo ? int(q_size[2]) : 0, int(hkv), int(d), rotate ? &plan.r : nullptr,
                              place.handle());
  });
  if (qo) return out.take();
  Py_RETURN_NONE;
}

// q [b, hq, d] and the pages of its sequences.
struct PagedInputs {
  const void* q;
  const int* lengths;
  at::IntArrayRef q_size;
  int b, hq, hkv, d;
  int64_t q_batch;
  Pages pages;
};
PagedInputs read_paged(Args& a, Place& place) {
  PagedInputs r;
  const at::Tensor& q = place.on(tensor("q", a.next(), at::kBFloat16));
  if (q.dim() != 3) value_error("q must be [b, hq, d]");
  sizes_fit(q);
  r.q_size = q.sizes();
  const auto qs = q.strides();
  if (qs[2] != 1 || (q.size(1) > 1 && qs[1] != q.size(2))) value_error("q's heads and features must be contiguous");
  r.q = q.data_ptr();
  r.b = int(q.size(0));
  r.hq = int(q.size(1));
  r.d = int(q.size(2));
  r.q_batch = used(q.size(0), qs[0]);
  r.pages = read_pages(a, r.d, place);
  r.hkv = int(r.pages.hkv);
  r.lengths = static_cast<const int*>(dense("lengths", a.next(), at::kInt, {r.b}, place).data_ptr());
  if (r.pages.rows != r.b) value_error(text("tables has ", r.pages.rows, " rows for ", r.b, " sequences"));
  return r;
}

PyObject* decode_paged(Args& a) {
  const Calls& calls = a.calls();
  Place place;
  const PagedInputs in = read_paged(a, place);
  const int window = a.keys(), sinks = a.keys();
  const float scale = a.scale();
  Out o = out_dense("o", a.next_or_none(), in.q_size, at::kBFloat16, place);
  Out lse = out_dense("lse", a.next_or_none(), {in.b, in.hq}, at::kFloat, place);
  Workspace ws;
  PyObject* given = a.next_or_none();
  if (given) ws.given(given, place);
  place.stream(a.next_or_none());
  make(o, in.q_size, at::kBFloat16, place);
  make(lse, {in.b, in.hq}, at::kFloat, place);
  // a shape that the call refuses needs none
  if (!given && in.pages.cap <= INT_MAX)
    ws.make(calls.decode_paged_bytes(in.b, in.hq, in.hkv, in.d, int(in.pages.cap), window, sinks), place);
  launch([&] {
    return calls.decode_paged(in.q, &in.pages.p, in.lengths, o.data(), static_cast<float*>(lse.data()), ws.data, ws.bytes,
                              in.b, in.hq, in.hkv, in.d, in.q_batch, window, sinks, scale, place.handle());
  });
  return results({&o, &lse});
}

PyObject* decode_shared(Args& a) {
  const Calls& calls = a.calls();
  Place place;
  const PagedInputs in = read_paged(a, place);
  const at::Tensor& shared = dense("shared", a.next(), at::kInt, place);
  if (shared.dim() != 1 || shared.size(0) < 1 || shared.size(0) > INT_MAX) value_error("shared must hold a count for each group");
  const int groups = int(shared.size(0));
  PyObject* offo = a.next_or_none();
  const int* offsets = nullptr;
  if (offo)
    offsets = static_cast<const int*>(dense("group_offsets", offo, at::kInt, {int64_t(groups) + 1}, place).data_ptr());
  else if (groups != 1)
    value_error(text("shared holds ", groups, " counts; without group_offsets the batch is one group"));
  PyObject* most = a.next_or_none();
  const int max_group = most ? int(Args::integer_of(most, "max_group")) : in.b;
  const float scale = a.scale();
  Out o = out_dense("o", a.next_or_none(), in.q_size, at::kBFloat16, place);
  Out lse = out_dense("lse", a.next_or_none(), {in.b, in.hq}, at::kFloat, place);
  Workspace ws;
  PyObject* given = a.next_or_none();
  if (given) ws.given(given, place);
  place.stream(a.next_or_none());
  make(o, in.q_size, at::kBFloat16, place);
  make(lse, {in.b, in.hq}, at::kFloat, place);
  if (!given) {
    // a shape that the call refuses needs none
    const size_t need = calls.decode_shared_bytes(in.b, in.hq, in.hkv, in.d, groups, max_group);
    ws.make(need > 0 ? need : 16, place);
  }
  launch([&] {
    return calls.decode_shared(in.q, &in.pages.p, in.lengths, shared.const_data_ptr<int>(), offsets, groups, max_group,
                               o.data(), static_cast<float*>(lse.data()), ws.data, ws.bytes, in.b, in.hq, in.hkv, in.d,
                               in.q_batch, scale, place.handle());
  });
  return results({&o, &lse});
}

// Runs a call; an error code of the library is returned as an int, which the
// Python side raises as CpattnError.
template <PyObject* (*F)(Args&)>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    Args a{args, n};
    return F(a);
  } catch (const Refused& e) {
    if (e.type) PyErr_SetString(e.type, e.what.c_str());
    return nullptr;
  } catch (const Failed& e) {
    return PyLong_FromLong(e.rc);
  }
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(Args&)>
constexpr PyCFunction method() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<F>));
}

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
  static PyMethodDef methods[] = {{"rope", method<rope>(), METH_FASTCALL, nullptr},
                                  {"qk_norm_rope", method<qk_norm_rope>(), METH_FASTCALL, nullptr},
                                  {"qk_norm_rope_bwd", method<qk_norm_rope_bwd>(), METH_FASTCALL, nullptr},
                                  {"fwd_window", method<fwd_window>(), METH_FASTCALL, nullptr},
                                  {"fwd_window_varlen", method<fwd_window_varlen>(), METH_FASTCALL, nullptr},
                                  {"bwd_window", method<bwd_window>(), METH_FASTCALL, nullptr},
                                  {"bwd_window_varlen", method<bwd_window_varlen>(), METH_FASTCALL, nullptr},
                                  {"decode", method<decode>(), METH_FASTCALL, nullptr},
                                  {"append_paged", method<append_paged>(), METH_FASTCALL, nullptr},
                                  {"decode_paged", method<decode_paged>(), METH_FASTCALL, nullptr},
                                  {"decode_shared", method<decode_shared>(), METH_FASTCALL, nullptr},
                                  {nullptr, nullptr, 0, nullptr}};
  static PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr,
                               nullptr};
  return PyModule_Create(&module);
}
