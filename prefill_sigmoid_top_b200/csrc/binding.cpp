// Argument marshalling of the calls whose GPU time is a few microseconds (routing from logits, the int8 products), as a
// CPython extension: checks of the tensors, the allocation of results and workspaces, the current stream, and the C
// entry point.  Marshalled in Python over ctypes these calls took 11 to 18 us of host time for 3 to 20 us on the GPU.
// No arithmetic and no kernel is here; what is refused, and how, is the Python wrappers' documentation.
//
// Every function returns its result, or the status of the C entry point as an int (the wrapper raises it).
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "moe_b200.h"

namespace {

using at::Tensor;

struct Refused {  // becomes a ValueError
  std::string what;
};

[[noreturn]] void refuse(const std::string& what) { throw Refused{what}; }

// The arguments of one call, in order.
struct Args {
  PyObject* const* a;
  Py_ssize_t n, at = 0;
  int device = -1;

  PyObject* next() {
    if (at >= n) refuse("too few arguments");
    return a[at++];
  }
  // A CUDA tensor on the device of the first one, or null for None.
  const Tensor* tensor_or_none() {
    PyObject* o = next();
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) refuse("expected a tensor");
    const Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda()) refuse("moe_b200 operates on CUDA tensors only");
    const int d = t.get_device();
    if (device < 0) device = d;
    if (d != device) refuse("tensors on different devices");
    return &t;
  }
  const Tensor& tensor(const char* what) {
    const Tensor* t = tensor_or_none();
    if (t == nullptr) refuse(std::string("no ") + what);
    return *t;
  }
  int64_t integer() {
    const long long v = PyLong_AsLongLong(next());
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
  }
  int32_t integer32() {
    const int64_t v = integer();
    if (v < INT32_MIN || v > INT32_MAX) refuse("integer out of range");
    return static_cast<int32_t>(v);
  }
  double real() {
    const double v = PyFloat_AsDouble(next());
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return v;
  }
  bool truth() {
    const int v = PyObject_IsTrue(next());
    if (v < 0) throw python_error();
    return v != 0;
  }
};

std::string shape_text(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + ")";
}

// A contiguous tensor of this type and shape.
const Tensor& want(const Tensor& t, at::ScalarType type, at::IntArrayRef shape, const char* what) {
  if (t.scalar_type() != type || t.sizes() != shape || !t.is_contiguous())
    refuse(std::string(what) + ": expected a contiguous " + c10::toString(type) + " tensor of shape " +
           shape_text(shape));
  return t;
}

void* address(const Tensor* t) { return t == nullptr ? nullptr : t->data_ptr(); }

// [rows, cols] with contiguous rows; the elements between rows (any value fits a single row).
int64_t row_stride(const Tensor& t, const char* what) {
  if (t.dim() != 2 || (t.size(1) > 1 && t.stride(1) != 1))
    refuse(std::string(what) + ": expected a tensor of two dimensions with contiguous rows");
  return t.size(0) > 1 ? t.stride(0) : t.size(1);
}

Tensor bytes_like(const Tensor& t, size_t n) {
  return at::empty({static_cast<int64_t>(n)}, t.options().dtype(at::kByte));
}

PyObject* wrap(const Tensor& t) { return THPVariable_Wrap(t); }

template <class F>
PyObject* guarded(F f) {
  HANDLE_TH_ERRORS
  try {
    return f();
  } catch (const Refused& r) {
    PyErr_SetString(PyExc_ValueError, r.what.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// logits, bias, top_k, n_group, topk_group, group_score, scoring, renormalize, routed_scale, topk_ids, topk_w
PyObject* route_logits(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args in{a, n};
    const Tensor& logits = in.tensor("logits");
    const int64_t ld = row_stride(logits, "logits");
    const at::ScalarType type = logits.scalar_type();
    if (type != at::kFloat && type != at::kBFloat16) refuse("logits: expected fp32 or bf16");
    const int64_t M = logits.size(0), E = logits.size(1);
    if (M > INT32_MAX || E > INT32_MAX) refuse("logits: too large");
    const Tensor* bias = in.tensor_or_none();
    if (bias) want(*bias, at::kFloat, {E}, "bias");
    const int32_t K = in.integer32();
    moe_group_opts_t o{};
    o.n_group = in.integer32();
    o.topk_group = in.integer32();
    o.group_score = in.integer32();
    o.scoring = in.integer32();
    o.renormalize = in.truth() ? 1 : 0;
    o.routed_scale = static_cast<float>(in.real());
    const Tensor* ids_in = in.tensor_or_none();
    const Tensor* w_in = in.tensor_or_none();
    const int64_t k = K < 0 || K > E ? 0 : K;  // what the entry point refuses gets no memory
    if (ids_in) want(*ids_in, at::kInt, {M, k}, "topk_ids");
    if (w_in) want(*w_in, at::kFloat, {M, k}, "topk_w");
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(in.device));
    const Tensor ids = ids_in ? *ids_in : at::empty({M, k}, logits.options().dtype(at::kInt));
    const Tensor w = w_in ? *w_in : at::empty({M, k}, logits.options().dtype(at::kFloat));
    const moe_status_t st = moe_route_logits(
        logits.data_ptr(), type == at::kFloat ? MOE_DT_F32 : MOE_DT_BF16, ld, static_cast<const float*>(address(bias)),
        static_cast<int32_t>(M), static_cast<int32_t>(E), K, &o, static_cast<int32_t*>(ids.data_ptr()),
        static_cast<float*>(w.data_ptr()), c10::cuda::getCurrentCUDAStream(in.device).stream());
    if (st != MOE_OK) return PyLong_FromLong(st);
    PyObject* r = PyTuple_New(2);
    if (r == nullptr) throw python_error();
    PyTuple_SET_ITEM(r, 0, wrap(ids));
    PyTuple_SET_ITEM(r, 1, wrap(w));
    return r;
  });
}

// The error word (nullable).
int32_t* read_err_flag(Args& in) {
  const Tensor* t = in.tensor_or_none();
  if (t == nullptr) return nullptr;
  want(*t, at::kInt, t->sizes(), "err_flag");
  if (t->numel() < 1) refuse("err_flag: expected at least one int32");
  return static_cast<int32_t*>(t->data_ptr());
}

// x, codes, scales, out, out_dtype, ws, err_flag
PyObject* linear_int8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args in{a, n};
    const Tensor& x = in.tensor("x");
    const int64_t ldx = row_stride(x, "x");
    if (x.scalar_type() != at::kBFloat16) refuse("x: expected bf16");
    const Tensor& codes = in.tensor("codes");
    const int64_t ld_codes = row_stride(codes, "codes");
    const int64_t M = x.size(0), K = x.size(1), N = codes.size(0);
    if (codes.scalar_type() != at::kChar || codes.size(1) != K) refuse("codes: expected an int8 [N, K] tensor");
    const int64_t ldw = N > 1 ? ld_codes : (K + 15) / 16 * 16;
    const Tensor& scales = want(in.tensor("scales"), at::kFloat, {N}, "scales");
    const Tensor* out_in = in.tensor_or_none();
    PyObject* dt = in.next();
    at::ScalarType type;
    if (out_in != nullptr) {
      if (out_in->dim() != 2 || out_in->size(0) != M || out_in->size(1) != N) refuse("out: expected [M, N]");
      type = out_in->scalar_type();
    } else {
      if (!THPDtype_Check(dt)) refuse("out_dtype: expected a torch.dtype");
      type = reinterpret_cast<THPDtype*>(dt)->scalar_type;
    }
    if (type != at::kFloat && type != at::kBFloat16) refuse("out: expected bf16 or fp32");
    const Tensor* ws_in = in.tensor_or_none();
    int32_t* err = read_err_flag(in);
    if (ws_in && !ws_in->is_contiguous()) refuse("ws: expected a contiguous tensor");
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(in.device));
    const Tensor out = out_in ? *out_in : at::empty({M, N}, x.options().dtype(type));
    const int64_t ldo = row_stride(out, "out");
    Tensor ws;
    size_t ws_bytes = 0;
    if (ws_in) {
      ws = *ws_in;
      ws_bytes = static_cast<size_t>(ws.nbytes());
    } else if ((ws_bytes = moe_linear_int8_workspace_size(M, N, K)) != 0) {
      ws = bytes_like(x, ws_bytes);
    }
    const moe_status_t st = moe_linear_int8(
        static_cast<const moe_bf16_t*>(x.data_ptr()), ldx, static_cast<const int8_t*>(codes.data_ptr()), ldw,
        static_cast<const float*>(scales.data_ptr()), M, N, K, out.data_ptr(), ldo,
        type == at::kFloat ? MOE_DT_F32 : MOE_DT_BF16, ws.defined() ? ws.data_ptr() : nullptr, ws_bytes,
        err, c10::cuda::getCurrentCUDAStream(in.device).stream());
    return st != MOE_OK ? PyLong_FromLong(st) : wrap(out);
  });
}

// The plan's arrays, each with as many entries as moe_align_block_size writes for this shape (more are fine, as buffers
// kept for a larger one have).  A shape that the library refuses has no capacity, and its call launches nothing.
moe_plan_t read_plan(Args& in, const moe_shape_t& s, int64_t cap) {
  const int64_t blocks = cap > 0 ? cap / s.block_size : 0;
  const struct {
    const char* name;
    int64_t entries;
  } arrays[5] = {{"sorted_ids", cap},
                 {"block_expert", blocks},
                 {"expert_counts", s.E},
                 {"expert_offsets", int64_t{s.E} + 1},
                 {"num_tokens_post_padded", 1}};
  const int32_t* p[5];
  for (int i = 0; i < 5; ++i) {
    const Tensor& t = in.tensor("plan");
    want(t, at::kInt, t.sizes(), "plan");
    if (t.numel() < arrays[i].entries)
      refuse(std::string("plan: ") + arrays[i].name + " has " + std::to_string(t.numel()) + " entries, the shape needs " +
             std::to_string(arrays[i].entries));
    p[i] = static_cast<const int32_t*>(t.data_ptr());
  }
  return {p[0], p[1], p[2], p[3], p[4]};
}
moe_shape_t read_shape(Args& in) {
  moe_shape_t s{};
  s.M = in.integer32();
  s.H = in.integer32();
  s.I = in.integer32();
  s.E = in.integer32();
  s.top_k = in.integer32();
  s.block_size = in.integer32();
  return s;
}
// codes [E, rows, cols] and scales [E, rows]
void read_matrix(Args& in, const char* name, int64_t E, int64_t rows, int64_t cols, const void** codes,
                 const float** scales) {
  const Tensor* c = in.tensor_or_none();
  const Tensor* s = in.tensor_or_none();
  if (c == nullptr || s == nullptr) refuse(std::string("Int8Weights without ") + name);
  *codes = want(*c, at::kChar, {E, rows, cols}, name).data_ptr();
  *scales = static_cast<const float*>(want(*s, at::kFloat, {E, rows}, (std::string(name) + "_scales").c_str()).data_ptr());
}
Tensor workspace(const Tensor* given, const Tensor& like, size_t need) {
  if (given == nullptr) return bytes_like(like, need ? need : 1);
  if (!given->is_contiguous()) refuse("ws: expected a contiguous tensor");
  return *given;
}

// x, shape (6), gate, gate_scales, up, up_scales, plan (5), h, err_flag, ws
PyObject* grouped_up_swiglu_int8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args in{a, n};
    const Tensor& x = in.tensor("x");
    const moe_shape_t s = read_shape(in);
    want(x, at::kBFloat16, {s.M, s.H}, "x");
    moe_weights_t w{};
    w.dtype = MOE_W_INT8;
    read_matrix(in, "gate", s.E, s.I, s.H, &w.gate, &w.gate_gs);
    read_matrix(in, "up", s.E, s.I, s.H, &w.up, &w.up_gs);
    const int64_t cap = static_cast<int64_t>(moe_align_capacity(s));
    const moe_plan_t plan = read_plan(in, s, cap);
    const Tensor* h_in = in.tensor_or_none();
    int32_t* err = read_err_flag(in);
    const Tensor* ws_in = in.tensor_or_none();
    if (h_in && (h_in->scalar_type() != at::kBFloat16 || !h_in->is_contiguous() || h_in->numel() < cap * s.I))
      refuse("h: expected align_capacity(shape) contiguous bf16 rows of I");
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(in.device));
    const Tensor h = h_in ? *h_in : at::empty({cap, s.I < 0 ? 0 : s.I}, x.options());
    const Tensor ws = workspace(ws_in, x, moe_up_workspace_size(s, MOE_W_INT8));
    const moe_status_t st = moe_grouped_up_swiglu(
        static_cast<const moe_bf16_t*>(x.data_ptr()), &w, &plan, s, static_cast<moe_bf16_t*>(h.data_ptr()),
        ws.data_ptr(), static_cast<size_t>(ws.nbytes()), err,
        c10::cuda::getCurrentCUDAStream(in.device).stream());
    return st != MOE_OK ? PyLong_FromLong(st) : wrap(h);
  });
}

// h, shape (6), down, down_scales, plan (5), y, err_flag, ws
PyObject* grouped_down_int8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Args in{a, n};
    const Tensor& h = in.tensor("h");
    const moe_shape_t s = read_shape(in);
    const int64_t cap = static_cast<int64_t>(moe_align_capacity(s));
    if (h.scalar_type() != at::kBFloat16 || !h.is_contiguous() || h.numel() < cap * s.I)
      refuse("h: expected align_capacity(shape) contiguous bf16 rows of I");
    moe_weights_t w{};
    w.dtype = MOE_W_INT8;
    read_matrix(in, "down", s.E, s.H, s.I, &w.down, &w.down_gs);
    const moe_plan_t plan = read_plan(in, s, cap);
    const Tensor* y_in = in.tensor_or_none();
    int32_t* err = read_err_flag(in);
    const Tensor* ws_in = in.tensor_or_none();
    const int64_t slots = static_cast<int64_t>(s.M) * s.top_k;
    if (y_in && (y_in->scalar_type() != at::kBFloat16 || !y_in->is_contiguous() || y_in->numel() != slots * s.H))
      refuse("y: expected M * top_k contiguous bf16 rows of H");
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(in.device));
    const Tensor y = y_in ? *y_in : at::empty({slots < 0 ? 0 : slots, s.H < 0 ? 0 : s.H}, h.options());
    const Tensor ws = workspace(ws_in, h, moe_down_workspace_size(s, MOE_W_INT8));
    const moe_status_t st = moe_grouped_down(
        static_cast<const moe_bf16_t*>(h.data_ptr()), &w, &plan, s, static_cast<moe_bf16_t*>(y.data_ptr()),
        ws.data_ptr(), static_cast<size_t>(ws.nbytes()), err,
        c10::cuda::getCurrentCUDAStream(in.device).stream());
    return st != MOE_OK ? PyLong_FromLong(st) : wrap(y);
  });
}

#define MOE_FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {MOE_FAST(route_logits), MOE_FAST(linear_int8), MOE_FAST(grouped_up_swiglu_int8),
                         MOE_FAST(grouped_down_int8), {nullptr, nullptr, 0, nullptr}};
#undef MOE_FAST

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
