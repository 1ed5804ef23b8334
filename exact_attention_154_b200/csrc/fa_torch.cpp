// fa_torch.cpp -- the torch side of the calls a model makes for every layer and
// token (norm and rotation, attention with a window and sinks, its gradient,
// its single-token form): argument checks, result tensors, the tensors' device
// and its current stream, then the C ABI of include/fa.h.
//
// Marshalling only, as fa.py's: every step runs in the library's kernels.  It is
// compiled because these calls are bound by the host where the work is small
// (measured on the token of eight sequences, 2.5 us on the GPU: 16.8 us a pass
// through ctypes, a third of it converting arguments).
#include <Python.h>
#include <dlfcn.h>

#include <ATen/ATen.h>
#include <ATen/MemoryOverlap.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "../../include/fa.h"

namespace {

decltype(&fa_qk_norm_rope) p_norm_rope = nullptr;
decltype(&fa_qk_norm_rope_bwd) p_norm_rope_bwd = nullptr;
decltype(&fa_fwd_sinks) p_fwd = nullptr;
decltype(&fa_bwd_sinks) p_bwd = nullptr;
decltype(&fa_bwd_sinks_workspace) p_bwd_workspace = nullptr;
decltype(&fa_decode_sinks) p_decode = nullptr;

// A refused argument: becomes Python's ValueError.
struct Refused {
  std::string what;
};
[[noreturn]] void refuse(const std::string& what) { throw Refused{what}; }

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a CUDA tensor");
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
  return t;
}

// A tensor on the device of the call's first one.
void same_device(const at::Tensor& t, const char* name, const at::Tensor& first) {
  if (t.device() != first.device())
    refuse(std::string(name) + " is on " + t.device().str() + ", expected " + first.device().str());
}

int dtype_code(const at::Tensor& t) { return t.scalar_type() == at::kBFloat16 ? FA_BF16 : FA_FP16; }

// A 16-bit CUDA tensor [B, H, N, d] whose rows are adjacent elements.
const at::Tensor& rows(PyObject* o, const char* name, const at::Tensor* first) {
  const at::Tensor& t = tensor(o, name);
  const auto st = t.scalar_type();
  if ((st != at::kBFloat16 && st != at::kHalf) || (first && st != first->scalar_type()))
    refuse(std::string(name) + " must be float16 or bfloat16, one type for all operands");
  if (t.dim() != 4 || t.stride(3) != 1)
    refuse(std::string(name) + " must be [B, H, N, d] with adjacent elements in a row");
  if (first) same_device(t, name, *first);
  return t;
}

// Whether the rows of [B, H, N, d] surely do not overlap: its dimensions,
// ordered by stride, each step over the one before.
bool fresh_rows(const at::Tensor& t) {
  int order[4] = {0, 1, 2, 3};
  for (int i = 1; i < 4; ++i)
    for (int j = i; j > 0 && t.stride(order[j]) < t.stride(order[j - 1]); --j)
      std::swap(order[j], order[j - 1]);
  int64_t need = 0;
  for (int i : order) {
    if (t.size(i) <= 1) continue;
    if (t.stride(i) <= need) return false;
    need += (t.size(i) - 1) * t.stride(i);
  }
  return true;
}

const long long* strides(const at::Tensor& t) {
  static_assert(sizeof(long long) == sizeof(int64_t), "strides are passed as they are");
  return t.is_contiguous() ? nullptr : reinterpret_cast<const long long*>(t.strides().data());
}

at::Tensor new_like(const at::Tensor& t) { return at::empty(t.sizes(), t.options()); }

int as_int(int64_t n) {
  if (n < INT32_MIN || n > INT32_MAX) refuse("a size does not fit 32 bits");
  return static_cast<int>(n);
}

// Refuses an output that lies over `in`: other blocks of the grid may still read there.
// The same elements in the same places are taken where a block reads all of its rows
// before it writes them (same_ok).  Only what is certain is refused: interleaved views,
// as of one packed projection, may be apart though their ranges meet.
void keep_apart(const at::Tensor& out, const char* name, const at::Tensor& in, const char* in_name,
                bool same_ok) {
  if (out.numel() == 0 || in.numel() == 0) return;  // (the library refuses those sizes)
  const bool at_start = out.data_ptr() == in.data_ptr();
  const bool same = at_start && out.sizes() == in.sizes() && out.strides() == in.strides();
  const auto overlap = at::get_overlap_status(out, in);
  if (same ? !same_ok
           : at_start || overlap == at::MemOverlapStatus::Partial || overlap == at::MemOverlapStatus::Full)
    refuse(std::string(name) + " overlaps " + in_name);
}

// `like`'s shape and type, contiguous, on its device.
const at::Tensor& contiguous_like(PyObject* o, const char* name, const at::Tensor& like) {
  const at::Tensor& t = tensor(o, name);
  if (t.sizes() != like.sizes() || t.scalar_type() != like.scalar_type())
    refuse(std::string(name) + " must match q");
  if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
  same_device(t, name, like);
  return t;
}

const at::Tensor& check_lse(PyObject* o, at::IntArrayRef sizes, const at::Tensor& first) {
  const at::Tensor& t = tensor(o, "lse");
  if (t.sizes() != sizes || t.scalar_type() != at::kFloat || !t.is_contiguous())
    refuse("lse must be a contiguous float32 tensor of q's shape without d");
  same_device(t, "lse", first);
  return t;
}

void* data(const at::Tensor& t) { return t.data_ptr(); }

// The call's device made current and its current stream.
struct OnDevice {
  c10::cuda::CUDAGuard guard;
  cudaStream_t stream;
  explicit OnDevice(const at::Tensor& t)
      : guard(t.device()), stream(c10::cuda::getCurrentCUDAStream(t.device().index())) {}
  CUstream_st* get() const { return reinterpret_cast<CUstream_st*>(stream); }
};

double number(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw python_error();
  return x;
}
int whole(PyObject* o) {
  const long long x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) throw python_error();
  return as_int(x);
}

int truth(PyObject* o) {
  const int x = PyObject_IsTrue(o);
  if (x < 0) throw python_error();
  return x;
}

// The result, or the library's status where it refused.
PyObject* status(int rc) { return PyLong_FromLong(rc); }
PyObject* wrap(const at::Tensor& t) { return THPVariable_Wrap(t); }
template <size_t N>
PyObject* tuple(PyObject* (&items)[N]) {
  PyObject* out = PyTuple_New(N);
  for (size_t i = 0; i < N; ++i) PyTuple_SET_ITEM(out, i, items[i]);
  return out;
}
PyObject* none() {
  Py_INCREF(Py_None);
  return Py_None;
}

void expect_args(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) refuse("wrong number of arguments");
  if (!p_decode) refuse("the library is not loaded");
}

// --------------------------------------------------- norm and rotation

struct Table {
  const at::Tensor *cos, *sin;
  const int* positions = nullptr;
  int max_pos, rot;
};
Table table(PyObject* cos, PyObject* sin, PyObject* positions, const at::Tensor& q) {
  Table t;
  t.cos = &tensor(cos, "cos");
  t.sin = &tensor(sin, "sin");
  for (const at::Tensor* x : {t.cos, t.sin})
    if (x->dim() != 2 || x->scalar_type() != at::kFloat || !x->is_contiguous() ||
        x->sizes() != t.cos->sizes())
      refuse("cos and sin must be contiguous float32 [max_pos, rot / 2] tensors");
  same_device(*t.cos, "cos", q);
  same_device(*t.sin, "sin", q);
  if (positions != Py_None) {
    const at::Tensor& p = tensor(positions, "positions");
    if (p.dim() != 2 || p.size(0) != q.size(0) || p.size(1) != q.size(2) ||
        p.scalar_type() != at::kInt || !p.is_contiguous())
      refuse("positions must be a contiguous int32 [B, N] tensor");
    same_device(p, "positions", q);
    t.positions = static_cast<const int*>(data(p));
  }
  t.max_pos = as_int(t.cos->size(0));
  t.rot = as_int(2 * t.cos->size(1));
  return t;
}

// Norm weights (or null): [d], of the operands' type or float32, both of one type.
struct Weights {
  const at::Tensor* w[2] = {nullptr, nullptr};
  int code;
  const void* ptr(int i) const { return w[i] ? data(*w[i]) : nullptr; }
};
Weights weights(PyObject* qw, PyObject* kw, const at::Tensor& q) {
  Weights r;
  r.code = dtype_code(q);
  const char* names[2] = {"q_weight", "k_weight"};
  PyObject* given[2] = {qw, kw};
  c10::optional<at::ScalarType> type;
  for (int i = 0; i < 2; ++i) {
    if (given[i] == Py_None) continue;
    const at::Tensor& t = tensor(given[i], names[i]);
    if (t.dim() != 1 || t.size(0) != q.size(3) || !t.is_contiguous() ||
        (t.scalar_type() != q.scalar_type() && t.scalar_type() != at::kFloat) ||
        (type && *type != t.scalar_type()))
      refuse("q_weight and k_weight must be contiguous [d] tensors of the operands' type or "
             "float32, both of one type");
    same_device(t, names[i], q);
    type = t.scalar_type();
    r.w[i] = &t;
    if (*type == at::kFloat) r.code = FA_FP32;
  }
  return r;
}

const at::Tensor& keys_of(PyObject* o, const char* name, const at::Tensor& q) {
  const at::Tensor& k = rows(o, name, &q);
  if (k.size(0) != q.size(0) || k.size(2) != q.size(2) || k.size(3) != q.size(3))
    refuse(std::string(name) + " must be [B, Hk, N, d] with q's B, N and d");
  return k;
}

at::Tensor output(PyObject* o, const char* name, const at::Tensor& like) {
  if (o == Py_None) return new_like(like);
  const at::Tensor& t = rows(o, name, &like);
  if (t.sizes() != like.sizes() || !fresh_rows(t))
    refuse(std::string(name) + " must have its input's shape and rows that do not overlap");
  return t;
}

// (q, k, cos, sin, positions, q_weight, k_weight, eps, interleaved, q_out, k_out)
PyObject* norm_rope(PyObject* const* a, Py_ssize_t n) {
  expect_args(n, 11);
  const at::Tensor& q = rows(a[0], "q", nullptr);
  const at::Tensor& k = keys_of(a[1], "k", q);
  const Table t = table(a[2], a[3], a[4], q);
  const Weights w = weights(a[5], a[6], q);
  const at::Tensor qo = output(a[9], "q_out", q), ko = output(a[10], "k_out", k);
  if (a[9] != Py_None) {
    keep_apart(qo, "q_out", q, "q", true);
    keep_apart(qo, "q_out", k, "k", false);
  }
  if (a[10] != Py_None) {
    keep_apart(ko, "k_out", k, "k", true);
    keep_apart(ko, "k_out", q, "q", false);
  }
  if (a[9] != Py_None && a[10] != Py_None) keep_apart(qo, "q_out", ko, "k_out", false);
  const OnDevice on(q);
  const int rc = p_norm_rope(
      data(q), data(k), data(qo), data(ko), strides(q), strides(k), strides(qo), strides(ko),
      static_cast<const float*>(data(*t.cos)), static_cast<const float*>(data(*t.sin)), t.positions,
      t.max_pos, w.ptr(0), w.ptr(1), w.code, static_cast<float>(number(a[7])), as_int(q.size(0)),
      as_int(q.size(1)), as_int(k.size(1)), as_int(q.size(2)), as_int(q.size(3)), t.rot,
      truth(a[8]), dtype_code(q), on.get());
  if (rc != FA_OK) return status(rc);
  PyObject* out[2] = {wrap(qo), wrap(ko)};
  return tuple(out);
}

// (dq_out, dk_out, q, k, cos, sin, positions, q_weight, k_weight, eps, interleaved)
PyObject* norm_rope_bwd(PyObject* const* a, Py_ssize_t n) {
  expect_args(n, 11);
  const at::Tensor& q = rows(a[2], "q", nullptr);
  const at::Tensor& k = keys_of(a[3], "k", q);
  const at::Tensor& gq = rows(a[0], "dq_out", &q);
  const at::Tensor& gk = rows(a[1], "dk_out", &q);
  if (gq.sizes() != q.sizes() || gk.sizes() != k.sizes())
    refuse("dq_out and dk_out must have the shapes of q and k");
  const Table t = table(a[4], a[5], a[6], q);
  const Weights w = weights(a[7], a[8], q);
  const at::Tensor dq = new_like(q), dk = new_like(k);
  at::Tensor dw[2];
  for (int i = 0; i < 2; ++i)
    if (w.w[i]) dw[i] = new_like(*w.w[i]);
  const at::Tensor ws = at::empty({FA_NORM_ROPE_PARTS, q.size(3)}, t.cos->options());
  const OnDevice on(q);
  const int rc = p_norm_rope_bwd(
      data(gq), data(gk), data(q), data(k), data(dq), data(dk), w.w[0] ? data(dw[0]) : nullptr,
      w.w[1] ? data(dw[1]) : nullptr, strides(gq), strides(gk), strides(q), strides(k),
      static_cast<const float*>(data(*t.cos)), static_cast<const float*>(data(*t.sin)), t.positions,
      t.max_pos, w.ptr(0), w.ptr(1), w.code, static_cast<float>(number(a[9])),
      static_cast<float*>(data(ws)), as_int(q.size(0)), as_int(q.size(1)), as_int(k.size(1)),
      as_int(q.size(2)), as_int(q.size(3)), t.rot, truth(a[10]), dtype_code(q), on.get());
  if (rc != FA_OK) return status(rc);
  PyObject* out[4] = {wrap(dq), wrap(dk), w.w[0] ? wrap(dw[0]) : none(), w.w[1] ? wrap(dw[1]) : none()};
  return tuple(out);
}

// --------------------------------------------------- window and sinks

// Checks of [B, Hk, N, d] keys and values against q's batch, last size and heads.
void check_kv(const at::Tensor& k, const at::Tensor& v, int64_t B, int64_t H, int64_t N, int64_t d) {
  if (k.sizes() != v.sizes() || k.size(0) != B || k.size(2) != N || k.size(3) != d ||
      k.size(1) < 1 || H % k.size(1) != 0)
    refuse("k and v must be [B, Hk, rows, d] with q's B and d (and N), H a multiple of Hk");
}
// An attention's given output against its inputs.
void apart_from(const at::Tensor& o, const at::Tensor& q, const at::Tensor& k, const at::Tensor& v) {
  keep_apart(o, "out", q, "q", true);
  keep_apart(o, "out", k, "k", false);
  keep_apart(o, "out", v, "v", false);
}
float scale_of(PyObject* o) { return o == Py_None ? 0.f : static_cast<float>(number(o)); }

// (q, k, v, window, sinks, scale, out, lse, return_lse)
PyObject* fwd_sinks(PyObject* const* a, Py_ssize_t n) {
  expect_args(n, 9);
  const at::Tensor& q = rows(a[0], "q", nullptr);
  const at::Tensor& k = rows(a[1], "k", &q);
  const at::Tensor& v = rows(a[2], "v", &q);
  check_kv(k, v, q.size(0), q.size(1), q.size(2), q.size(3));
  const int window = whole(a[3]), sinks = whole(a[4]);
  const at::Tensor o = a[6] == Py_None ? new_like(q) : contiguous_like(a[6], "out", q);
  if (a[6] != Py_None) apart_from(o, q, k, v);
  const int with_lse = truth(a[8]);
  at::Tensor lse;
  if (with_lse)
    lse = a[7] == Py_None ? at::empty(q.sizes().slice(0, 3), q.options().dtype(at::kFloat))
                          : check_lse(a[7], q.sizes().slice(0, 3), q);
  const OnDevice on(q);
  const int rc = p_fwd(data(q), data(k), data(v), data(o),
                       with_lse ? static_cast<float*>(data(lse)) : nullptr, strides(q), strides(k),
                       strides(v), as_int(q.size(0)), as_int(q.size(1)), as_int(k.size(1)),
                       as_int(q.size(2)), as_int(q.size(3)), window, sinks, scale_of(a[5]),
                       dtype_code(q), on.get());
  if (rc != FA_OK) return status(rc);
  PyObject* out[2] = {wrap(o), with_lse ? wrap(lse) : none()};
  return tuple(out);
}

// (q, k, v, o, lse, dout, window, sinks, scale)
PyObject* bwd_sinks(PyObject* const* a, Py_ssize_t n) {
  expect_args(n, 9);
  const at::Tensor& q = rows(a[0], "q", nullptr);
  const at::Tensor& k = rows(a[1], "k", &q);
  const at::Tensor& v = rows(a[2], "v", &q);
  check_kv(k, v, q.size(0), q.size(1), q.size(2), q.size(3));
  const at::Tensor& o = contiguous_like(a[3], "o", q);
  const at::Tensor& lse = check_lse(a[4], q.sizes().slice(0, 3), q);
  const at::Tensor& g = contiguous_like(a[5], "dout", q);
  const int window = whole(a[6]), sinks = whole(a[7]);
  const int B = as_int(q.size(0)), H = as_int(q.size(1)), Hk = as_int(k.size(1)),
            N = as_int(q.size(2)), d = as_int(q.size(3));
  const long long floats = p_bwd_workspace(B, H, Hk, N, d, window, sinks);
  if (floats < 0) return status(static_cast<int>(floats));
  const at::Tensor dq = new_like(q), dk = new_like(k), dv = new_like(v);
  const at::Tensor ws = at::empty({floats}, lse.options());
  const OnDevice on(q);
  const int rc = p_bwd(data(q), data(k), data(v), data(o), static_cast<const float*>(data(lse)),
                       data(g), data(dq), data(dk), data(dv), strides(q), strides(k), strides(v),
                       static_cast<float*>(data(ws)), B, H, Hk, N, d, window, sinks, scale_of(a[8]),
                       dtype_code(q), on.get());
  if (rc != FA_OK) return status(rc);
  PyObject* out[3] = {wrap(dq), wrap(dk), wrap(dv)};
  return tuple(out);
}

// (q, k, v, seqlens, window, sinks, scale, out, return_lse)
PyObject* decode_sinks(PyObject* const* a, Py_ssize_t n) {
  expect_args(n, 9);
  const at::Tensor& q = tensor(a[0], "q");
  if (q.scalar_type() != at::kBFloat16 && q.scalar_type() != at::kHalf)
    refuse("q must be float16 or bfloat16");
  if (q.dim() != 3 || !q.is_contiguous()) refuse("q must be contiguous [B, H, d]");
  const at::Tensor& k = rows(a[1], "k", &q);
  const at::Tensor& v = rows(a[2], "v", &q);
  check_kv(k, v, q.size(0), q.size(1), k.size(2), q.size(2));
  const at::Tensor& lens = tensor(a[3], "seqlens");
  if (lens.dim() != 1 || lens.size(0) != q.size(0) || lens.scalar_type() != at::kInt ||
      !lens.is_contiguous())
    refuse("seqlens must be a contiguous int32 [B] tensor");
  same_device(lens, "seqlens", q);
  const int window = whole(a[4]), sinks = whole(a[5]);
  const at::Tensor o = a[7] == Py_None ? new_like(q) : contiguous_like(a[7], "out", q);
  if (a[7] != Py_None) apart_from(o, q, k, v);
  const int with_lse = truth(a[8]);
  at::Tensor lse;
  if (with_lse) lse = at::empty(q.sizes().slice(0, 2), q.options().dtype(at::kFloat));
  const OnDevice on(q);
  const int rc = p_decode(data(q), data(k), data(v), data(o),
                          with_lse ? static_cast<float*>(data(lse)) : nullptr,
                          static_cast<const int*>(data(lens)), strides(k), strides(v),
                          as_int(q.size(0)), as_int(q.size(1)), as_int(k.size(1)), as_int(k.size(2)),
                          as_int(q.size(2)), window, sinks, scale_of(a[6]), dtype_code(q), on.get());
  if (rc != FA_OK) return status(rc);
  PyObject* out[2] = {wrap(o), with_lse ? wrap(lse) : none()};
  return tuple(out);
}

// ------------------------------------------------------------- module

template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    return F(args, n);
  } catch (const Refused& r) {
    PyErr_SetString(PyExc_ValueError, r.what.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// load(path): resolves the entry points in the library at `path`.
PyObject* load(PyObject*, PyObject* path) {
  const char* s = PyUnicode_AsUTF8(path);
  if (!s) return nullptr;
  void* lib = dlopen(s, RTLD_NOW | RTLD_LOCAL);
  if (!lib) return PyErr_Format(PyExc_RuntimeError, "%s", dlerror());
  auto find = [&](auto& fn, const char* name) {
    fn = reinterpret_cast<std::decay_t<decltype(fn)>>(dlsym(lib, name));
    if (!fn) PyErr_Format(PyExc_RuntimeError, "%s lacks %s", s, name);
    return fn != nullptr;
  };
  if (!find(p_norm_rope, "fa_qk_norm_rope") || !find(p_norm_rope_bwd, "fa_qk_norm_rope_bwd") ||
      !find(p_fwd, "fa_fwd_sinks") || !find(p_bwd, "fa_bwd_sinks") ||
      !find(p_bwd_workspace, "fa_bwd_sinks_workspace") || !find(p_decode, "fa_decode_sinks"))
    return nullptr;
  return none();
}

#define FA_METHOD(name, fn) \
  {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&call<fn>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FA_METHOD("qk_norm_rope", norm_rope),
                         FA_METHOD("qk_norm_rope_bwd", norm_rope_bwd),
                         FA_METHOD("fwd_sinks", fwd_sinks),
                         FA_METHOD("bwd_sinks", bwd_sinks),
                         FA_METHOD("decode_sinks", decode_sinks),
                         {"load", load, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fa_torch", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" PyMODINIT_FUNC PyInit__fa_torch() { return PyModule_Create(&module); }
