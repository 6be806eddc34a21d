// The torch side of the operators around the products: argument checks, output
// tensors and the current stream, then the C calls of dg.h.  dg.py's functions of
// the same names call these; in Python the same checks and allocations take as
// long again as the kernel launch (combine: 7.6 us a call, here 3.8).
#include <ATen/ATen.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/hip/HIPCachingAllocator.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <dlfcn.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <string>
#include <vector>

#include "dg.h"

namespace {

using at::Tensor;
using c10::ScalarType;

struct Library {
  decltype(&dg_moe_rows) moe_rows;
  decltype(&dg_moe_sort_workspace) moe_sort_workspace;
  decltype(&dg_moe_sort) moe_sort;
  decltype(&dg_moe_permute) moe_permute;
  decltype(&dg_moe_permute_fp8) moe_permute_fp8;
  decltype(&dg_moe_combine) moe_combine;
  decltype(&dg_moe_combine_bwd) moe_combine_bwd;
  decltype(&dg_swiglu_fp8) swiglu_fp8;
  decltype(&dg_swiglu_fp8_bwd) swiglu_fp8_bwd;
  decltype(&dg_grouped_wgrad_fp8) grouped_wgrad_fp8;
  // null where an earlier build of the library lacks them
  decltype(&dg_moe_route_workspace) moe_route_workspace;
  decltype(&dg_moe_route) moe_route;
  decltype(&dg_moe_route_bwd) moe_route_bwd;
  decltype(&dg_residual_norm) residual_norm;
  decltype(&dg_residual_norm_bwd_workspace) residual_norm_bwd_workspace;
  decltype(&dg_residual_norm_bwd) residual_norm_bwd;
  decltype(&dg_grad_norm_workspace) grad_norm_workspace;
  decltype(&dg_grad_norm) grad_norm;
  decltype(&dg_clip_grads) clip_grads;
} lib;
PyObject* dg_error = nullptr;      // dg.DGError

// ---- arguments ------------------------------------------------------------------

std::string name_of(ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "bfloat16";
    case at::kFloat: return "float32";
    case at::kInt: return "int32";
    case at::kLong: return "int64";
    case at::kByte: return "uint8";
    case at::kFloat8_e4m3fn: return "float8_e4m3fn";
    default: return c10::toString(t);
  }
}

std::string shape_of(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + (s.size() == 1 ? ",)" : ")");
}

// The Python error is set here and passed on by END_HANDLE_TH_ERRORS.
[[noreturn]] void raise(PyObject* type, const std::string& message) {
  PyErr_SetString(type, message.c_str());
  throw python_error();
}
[[noreturn]] void type_error(const std::string& m) { raise(PyExc_TypeError, m); }
[[noreturn]] void value_error(const std::string& m) { raise(PyExc_ValueError, m); }

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a tensor, got " + Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}

// `t` is a contiguous tensor on the current device, of one of `dtypes`.
void check(const Tensor& t, const char* name, std::initializer_list<ScalarType> dtypes) {
  bool known = false;
  for (ScalarType d : dtypes) known |= t.scalar_type() == d;
  if (!known) {
    std::string m = std::string(name) + " must be ";
    const char* sep = "";
    for (ScalarType d : dtypes) {
      m += sep + name_of(d);
      sep = " or ";
    }
    type_error(m + ", got " + name_of(t.scalar_type()));
  }
  if (!t.is_cuda() || !t.is_contiguous()) value_error(std::string(name) + " must be a contiguous device tensor");
  if (t.get_device() != c10::hip::current_device())
    value_error(std::string(name) + " is on " + t.device().str() + ", the current device is cuda:" +
                std::to_string(c10::hip::current_device()));
}

void check(const Tensor& t, const char* name, std::initializer_list<ScalarType> dtypes, at::IntArrayRef shape) {
  check(t, name, dtypes);
  if (t.sizes() != shape)
    value_error(std::string(name) + " has shape " + shape_of(t.sizes()) + ", expected " + shape_of(shape));
}

// A matrix of activations; its dg_in_dtype.
int check_values(const Tensor& t, const char* name) {
  if (t.dim() != 2) value_error(std::string(name) + " must be a 2-D tensor");
  check(t, name, {at::kBFloat16, at::kFloat});
  return t.scalar_type() == at::kBFloat16 ? DG_IN_BF16 : DG_IN_F32;
}

// top_k of a plan's map of T tokens.
int check_slots(const Tensor& slot_row, int64_t T) {
  if (slot_row.dim() != 2 || slot_row.size(0) != T || slot_row.size(1) < 1)
    value_error("slot_row has shape " + shape_of(slot_row.sizes()) + ", expected (" + std::to_string(T) + ", top_k)");
  check(slot_row, "slot_row", {at::kInt});
  return int(std::min<int64_t>(slot_row.size(1), INT32_MAX));
}

int64_t check_rows(const Tensor& row_slot) {
  if (row_slot.dim() != 1) value_error("row_slot must be a 1-D tensor");
  check(row_slot, "row_slot", {at::kInt});
  return row_slot.size(0);
}

// A new tensor on `like`'s device (at::empty without its dispatch, 0.3 us).
Tensor create(at::IntArrayRef shape, ScalarType dtype, const Tensor& like) {
  return at::detail::empty_cuda(shape, dtype, like.device(), c10::nullopt);
}

// The output `o`, checked, or a new tensor.  What is written counts as written:
// autograd then sees a saved tensor that has changed.
Tensor output(PyObject* o, const char* name, at::IntArrayRef shape, ScalarType dtype, const Tensor& like) {
  if (o == nullptr || o == Py_None) return create(shape, dtype, like);
  const Tensor& t = tensor(o, name);
  check(t, name, {dtype}, shape);
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
  return t;
}

// Elements from the `at`-th on of `whole`, as a tensor of their own.
Tensor part(const Tensor& whole, int64_t at, at::IntArrayRef sizes) {
  Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(whole.storage()), whole.key_set(), whole.dtype());
  t.unsafeGetTensorImpl()->set_storage_offset(at);
  t.unsafeGetTensorImpl()->set_sizes_contiguous(sizes);
  return t;
}

int64_t integer(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    type_error(std::string(name) + " must be an integer");
  }
  return v;
}

int small(PyObject* o, const char* name) {
  const int64_t v = integer(o, name);
  if (v < INT32_MIN || v > INT32_MAX) value_error(std::string(name) + " is out of range");
  return int(v);
}

void arguments(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) type_error("expected " + std::to_string(want) + " arguments, got " + std::to_string(n));
}

float real(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    type_error(std::string(name) + " must be a number");
  }
  return float(v);
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v != 0;
}

// The tensor `o`, checked, or null for None; its address.
const Tensor* optional(PyObject* o, const char* name) { return o == Py_None ? nullptr : &tensor(o, name); }
const float* weights_of(PyObject* o, const char* name, at::IntArrayRef shape) {
  const Tensor* t = optional(o, name);
  if (!t) return nullptr;
  check(*t, name, {at::kFloat}, shape);
  return static_cast<const float*>(t->data_ptr());
}

// One element on the device, whatever its dimensions.
const void* scalar(const Tensor& t, const char* name, ScalarType dtype) {
  check(t, name, {dtype});
  if (t.numel() != 1) value_error(std::string(name) + " must have one element");
  return t.data_ptr();
}

template <typename F>
void need(F f, const char* name) {
  if (!f) raise(PyExc_RuntimeError, std::string("the library lacks ") + name + ": build it again");
}

hipStream_t stream() { return c10::hip::getCurrentHIPStream().stream(); }

template <typename T>
T* data(const Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}

// ---- results --------------------------------------------------------------------

PyObject* failure(int64_t status, const char* call) {
  PyObject* e = PyObject_CallFunction(dg_error, "Ls", (long long)status, call);
  if (e) {
    PyErr_SetObject(dg_error, e);
    Py_DECREF(e);
  }
  return nullptr;
}

PyObject* wrap(const Tensor& t) {
  if (t.defined()) return THPVariable_Wrap(t);
  Py_RETURN_NONE;
}

template <typename... Ts>
PyObject* tuple(const Ts&... ts) {
  PyObject* r = PyTuple_New(sizeof...(ts));
  if (!r) return nullptr;
  Py_ssize_t i = 0;
  (PyTuple_SET_ITEM(r, i++, wrap(ts)), ...);
  return r;
}

// ---- the operators ----------------------------------------------------------------

// moe_sort(ids, num_groups, align, rows or None)
PyObject* moe_sort(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 4);
  const Tensor& ids = tensor(a[0], "ids");
  if (ids.dim() != 2) value_error("ids must be [T][top_k]");
  check(ids, "ids", {at::kInt, at::kLong});
  const int64_t T = ids.size(0), k = ids.size(1);
  const int G = small(a[1], "num_groups"), align = small(a[2], "align");
  // what the sort would refuse is refused before anything is allocated for it
  int64_t M = k > INT32_MAX ? int64_t(DG_ERR_INVALID_ARG) : lib.moe_rows(T, int(k), G, align);
  if (M < 0) return failure(M, "dg_moe_sort");
  const int64_t ws = lib.moe_sort_workspace(T, int(k), G);
  if (a[3] != Py_None) {
    const int64_t rows = integer(a[3], "rows");
    if (rows < M || rows % align != 0) return failure(DG_ERR_INVALID_ARG, "dg_moe_sort");
    M = rows;
  }
  if (M > INT32_MAX) return failure(DG_ERR_INVALID_ARG, "dg_moe_sort");
  // one allocation for the plan: four cost 2 us more
  const Tensor all = create({2 * int64_t(G) + 1 + M + T * k}, at::kInt, ids);
  const Tensor offs = part(all, 0, {G + 1}), counts = part(all, G + 1, {G});
  const Tensor row_slot = part(all, 2 * int64_t(G) + 1, {M});
  const Tensor slot_row = part(all, 2 * int64_t(G) + 1 + M, {T, k});
  // (the workspace is free for the stream's later work when the call returns)
  const Tensor work = ws ? create({ws}, at::kByte, ids) : Tensor();
  const int st = lib.moe_sort(ids.data_ptr(), ids.scalar_type() == at::kLong ? DG_IDX_I64 : DG_IDX_I32, T, int(k), G,
                              align, M, data<int32_t>(offs), data<int32_t>(counts), data<int32_t>(row_slot),
                              data<int32_t>(slot_row), ws ? work.data_ptr() : nullptr, stream());
  if (st != DG_OK) return failure(st, "dg_moe_sort");
  return tuple(offs, counts, row_slot, slot_row);
  END_HANDLE_TH_ERRORS
}

// moe_permute(X, slot_row, row_slot, Y)
PyObject* moe_permute(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 4);
  const Tensor &X = tensor(a[0], "X"), &slot_row = tensor(a[1], "slot_row"), &row_slot = tensor(a[2], "row_slot");
  const int code = check_values(X, "X");
  const int64_t T = X.size(0), H = X.size(1);
  const int k = check_slots(slot_row, T);
  const int64_t M = check_rows(row_slot);
  const Tensor Y = output(a[3], "Y", {M, H}, X.scalar_type(), X);
  const int st = lib.moe_permute(X.data_ptr(), code, Y.data_ptr(), data<int32_t>(slot_row), data<int32_t>(row_slot), T,
                                 k, M, H, stream());
  if (st != DG_OK) return failure(st, "dg_moe_permute");
  return wrap(Y);
  END_HANDLE_TH_ERRORS
}

// moe_permute_fp8(X, slot_row, row_slot, scale mode, Q, S)
PyObject* moe_permute_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 6);
  const Tensor &X = tensor(a[0], "X"), &slot_row = tensor(a[1], "slot_row"), &row_slot = tensor(a[2], "row_slot");
  const int code = check_values(X, "X"), mode = small(a[3], "scale");
  const int64_t T = X.size(0), H = X.size(1);
  const int k = check_slots(slot_row, T);
  const int64_t M = check_rows(row_slot);
  const Tensor Q = output(a[4], "Q", {M, H}, at::kByte, X);
  const Tensor S = output(a[5], "S", {M, (H + 127) / 128}, at::kFloat, X);
  const int st = lib.moe_permute_fp8(X.data_ptr(), code, Q.data_ptr(), data<float>(S), mode, data<int32_t>(slot_row),
                                     data<int32_t>(row_slot), T, k, M, H, stream());
  if (st != DG_OK) return failure(st, "dg_moe_permute_fp8");
  return tuple(Q, S);
  END_HANDLE_TH_ERRORS
}

// moe_combine(Y, slot_row, weights, out)
PyObject* moe_combine(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 4);
  const Tensor &Y = tensor(a[0], "Y"), &slot_row = tensor(a[1], "slot_row");
  const int code = check_values(Y, "Y");
  const int64_t M = Y.size(0), H = Y.size(1), T = slot_row.dim() > 0 ? slot_row.size(0) : 0;
  const int k = check_slots(slot_row, T);
  const float* w = nullptr;
  if (a[2] != Py_None) {
    const Tensor& weights = tensor(a[2], "weights");
    check(weights, "weights", {at::kFloat}, {T, k});
    w = data<float>(weights);
  }
  const Tensor out = output(a[3], "out", {T, H}, Y.scalar_type(), Y);
  const int st = lib.moe_combine(Y.data_ptr(), code, w, data<int32_t>(slot_row), out.data_ptr(), T, k, M, H, stream());
  if (st != DG_OK) return failure(st, "dg_moe_combine");
  return wrap(out);
  END_HANDLE_TH_ERRORS
}

// moe_combine_bwd(dOut, Y, slot_row, row_slot, weights, dY, dweights)
PyObject* moe_combine_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 7);
  const Tensor &dOut = tensor(a[0], "dOut"), &Y = tensor(a[1], "Y"), &slot_row = tensor(a[2], "slot_row"),
               &row_slot = tensor(a[3], "row_slot"), &weights = tensor(a[4], "weights");
  const int code = check_values(dOut, "dOut");
  const int64_t T = dOut.size(0), H = dOut.size(1);
  const int k = check_slots(slot_row, T);
  const int64_t M = check_rows(row_slot);
  check(Y, "Y", {dOut.scalar_type()}, {M, H});
  check(weights, "weights", {at::kFloat}, {T, k});
  const Tensor dY = output(a[5], "dY", {M, H}, dOut.scalar_type(), dOut);
  const Tensor dw = output(a[6], "dweights", {T, k}, at::kFloat, dOut);
  const int st = lib.moe_combine_bwd(dOut.data_ptr(), Y.data_ptr(), code, data<float>(weights), data<int32_t>(slot_row),
                                     data<int32_t>(row_slot), dY.data_ptr(), data<float>(dw), T, k, M, H, stream());
  if (st != DG_OK) return failure(st, "dg_moe_combine_bwd");
  return tuple(dY, dw);
  END_HANDLE_TH_ERRORS
}

// swiglu_fp8(H, checkpoint)
PyObject* swiglu_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 2);
  const Tensor& H = tensor(a[0], "H");
  const int code = check_values(H, "H");
  const int checkpoint = PyObject_IsTrue(a[1]);
  if (checkpoint < 0) return nullptr;
  if (H.size(1) % 2) value_error("H must have an even number of columns");
  const int64_t M = H.size(0), I = H.size(1) / 2, Ib = (I + 127) / 128;
  const Tensor A = create({M, I}, at::kByte, H);
  Tensor sA, Hq, sH;
  if (checkpoint) {
    // the scales, 1/32 of the codes' bytes, in one allocation (256 rows of 2 x 2048:
    // 6.4 us a call, with two 6.8); codes are of another type, which could not be
    // saved to a file together with scales in the same memory
    const Tensor scales = create({3 * M * Ib}, at::kFloat, H);
    sA = part(scales, 0, {M, Ib});
    sH = part(scales, M * Ib, {M, 2, Ib});
    Hq = create({M, 2 * I}, at::kByte, H);
  } else {
    sA = create({M, Ib}, at::kFloat, H);
  }
  // an empty checkpoint's addresses are null, which would ask for none: no work either way
  const int st = lib.swiglu_fp8(H.data_ptr(), code, A.data_ptr(), data<float>(sA), checkpoint ? Hq.data_ptr() : nullptr,
                                checkpoint ? data<float>(sH) : nullptr, M, I, stream());
  if (st != DG_OK) return failure(st, "dg_swiglu_fp8");
  return tuple(A, sA, Hq, sH);
  END_HANDLE_TH_ERRORS
}

// swiglu_fp8_bwd(dA, Hq, sH, dH)
PyObject* swiglu_fp8_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 4);
  const Tensor &dA = tensor(a[0], "dA"), &Hq = tensor(a[1], "Hq"), &sH = tensor(a[2], "sH");
  const int code = check_values(dA, "dA");
  const int64_t M = dA.size(0), I = dA.size(1);
  check(Hq, "Hq", {at::kByte, at::kFloat8_e4m3fn}, {M, 2 * I});
  check(sH, "sH", {at::kFloat}, {M, 2, (I + 127) / 128});
  const Tensor dH = output(a[3], "dH", {M, 2 * I}, dA.scalar_type(), dA);
  const int st = lib.swiglu_fp8_bwd(dA.data_ptr(), code, Hq.data_ptr(), data<float>(sH), dH.data_ptr(), M, I, stream());
  if (st != DG_OK) return failure(st, "dg_swiglu_fp8_bwd");
  return wrap(dH);
  END_HANDLE_TH_ERRORS
}

// grouped_wgrad_fp8(dY, X, sX, group_offsets, group_counts, out dtype, dW, accumulate)
PyObject* grouped_wgrad_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 8);
  const Tensor &dY = tensor(a[0], "dY"), &X = tensor(a[1], "X"), &sX = tensor(a[2], "sX"),
               &offs = tensor(a[3], "group_offsets");
  if (dY.dim() != 2 || X.dim() != 2 || offs.dim() != 1) value_error("dY and X must be 2-D, group_offsets 1-D");
  const int64_t M = dY.size(0), N = dY.size(1), K = X.size(1), G = offs.size(0) - 1;
  check(dY, "dY", {at::kBFloat16});
  check(X, "X", {at::kByte, at::kFloat8_e4m3fn}, {M, K});
  check(sX, "sX", {at::kFloat}, {M, (K + 127) / 128});
  check(offs, "group_offsets", {at::kInt});
  const int32_t* counts = nullptr;
  if (a[4] != Py_None) {
    const Tensor& t = tensor(a[4], "group_counts");
    check(t, "group_counts", {at::kInt}, {G});
    counts = data<int32_t>(t);
  }
  const int out = small(a[5], "out_dtype"), accumulate = PyObject_IsTrue(a[7]);
  if (accumulate < 0) return nullptr;
  if (accumulate && a[6] == Py_None) value_error("accumulate needs dW");
  if (G < 1 || G > INT32_MAX) value_error("group_offsets must have at least two entries");
  const Tensor dW = output(a[6], "dW", {G, N, K}, out == DG_OUT_F32 ? at::kFloat : at::kBFloat16, dY);
  const int st = lib.grouped_wgrad_fp8(dY.data_ptr(), X.data_ptr(), data<float>(sX), data<int32_t>(offs), counts,
                                       int(G), M, N, K, dW.data_ptr(), out, accumulate, stream());
  if (st != DG_OK) return failure(st, "dg_grouped_wgrad_fp8");
  return wrap(dW);
  END_HANDLE_TH_ERRORS
}

// moe_route(logits, top_k, score, renormalise, scale, bias, mask, balance)
PyObject* moe_route(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 8);
  need(lib.moe_route, "dg_moe_route");
  const Tensor& x = tensor(a[0], "logits");
  const int code = check_values(x, "logits"), k = small(a[1], "top_k"), score = small(a[2], "score");
  const bool renormalise = truth(a[3]), balance = truth(a[7]);
  const float scale = real(a[4], "scale");
  const int64_t T = x.size(0), E = x.size(1);
  const float* bias = weights_of(a[5], "bias", {E});
  const uint8_t* mask = nullptr;
  if (a[6] != Py_None) {
    const Tensor& m = tensor(a[6], "mask");
    check(m, "mask", {at::kBool, at::kByte}, {T});
    mask = static_cast<const uint8_t*>(m.data_ptr());
  }
  // what the call would refuse is refused before anything is allocated for it
  const int64_t ws = lib.moe_route_workspace(T, E, k);
  if (ws < 0) return failure(ws, "dg_moe_route");
  const Tensor ids = create({T, k}, at::kInt, x), weights = create({T, k}, at::kFloat, x);
  Tensor counts, sums, routed, loss;
  c10::DataPtr work;
  if (balance) {
    // the load in one allocation for each type; what the tokens have lies alone, so that
    // a loss that is kept keeps no batch alive (8192 tokens, 64 experts: 10.2 us of host time,
    // with three allocations in all 9.8).  The workspace, which no tensor needs to hold (0.3
    // us), is free for the stream's later work when the call returns
    const Tensor ints = create({E + 1}, at::kInt, x), floats = create({E + 1}, at::kFloat, x);
    counts = part(ints, 0, {E});
    routed = part(ints, E, {});
    sums = part(floats, 0, {E});
    loss = part(floats, E, {});
    if (ws) work = c10::hip::HIPCachingAllocator::get()->allocate(ws);
  }
  const int st = lib.moe_route(x.data_ptr(), code, bias, mask, T, E, k, score, renormalise, scale, data<int32_t>(ids),
                               data<float>(weights), balance ? data<int32_t>(counts) : nullptr,
                               balance ? data<float>(sums) : nullptr, balance ? data<int32_t>(routed) : nullptr,
                               balance ? data<float>(loss) : nullptr, work.get(), stream());
  if (st != DG_OK) return failure(st, "dg_moe_route");
  return tuple(ids, weights, counts, sums, routed, loss);
  END_HANDLE_TH_ERRORS
}

// moe_route_bwd(dweights, logits, ids, score, renormalise, scale, dloss, counts, routed, dlogits)
PyObject* moe_route_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 10);
  need(lib.moe_route_bwd, "dg_moe_route_bwd");
  const Tensor &dw = tensor(a[0], "dweights"), &x = tensor(a[1], "logits"), &ids = tensor(a[2], "ids");
  const int code = check_values(x, "logits"), score = small(a[3], "score");
  const bool renormalise = truth(a[4]);
  const float scale = real(a[5], "scale");
  const int64_t T = x.size(0), E = x.size(1);
  if (ids.dim() != 2 || ids.size(0) != T) value_error("ids has shape " + shape_of(ids.sizes()) + ", expected (" +
                                                      std::to_string(T) + ", top_k)");
  check(ids, "ids", {at::kInt});
  const int k = int(std::min<int64_t>(ids.size(1), INT32_MAX));
  check(dw, "dweights", {at::kFloat}, {T, k});
  const float* dloss = nullptr;
  const int32_t *counts = nullptr, *routed = nullptr;
  if (const Tensor* t = optional(a[6], "dloss")) {
    dloss = static_cast<const float*>(scalar(*t, "dloss", at::kFloat));
    if (a[7] == Py_None || a[8] == Py_None) value_error("dloss needs counts and routed");
    const Tensor &c = tensor(a[7], "counts"), &r = tensor(a[8], "routed");
    check(c, "counts", {at::kInt}, {E});
    counts = data<int32_t>(c);
    routed = static_cast<const int32_t*>(scalar(r, "routed", at::kInt));
  }
  const int64_t refused = lib.moe_route_workspace(T, E, k);
  if (refused < 0) return failure(refused, "dg_moe_route_bwd");
  const Tensor dx = output(a[9], "dlogits", {T, E}, x.scalar_type(), x);
  const int st = lib.moe_route_bwd(data<float>(dw), x.data_ptr(), code, data<int32_t>(ids), counts, routed, dloss, T, E,
                                   k, score, renormalise, scale, dx.data_ptr(), stream());
  if (st != DG_OK) return failure(st, "dg_moe_route_bwd");
  return wrap(dx);
  END_HANDLE_TH_ERRORS
}

int dtype_code(const Tensor& t) { return t.scalar_type() == at::kBFloat16 ? DG_IN_BF16 : DG_IN_F32; }

// A gate's kind by its shape: [H] by channel, [T][1] by token.
int gate_of(PyObject* o, int64_t T, int64_t H, const float** gate) {
  *gate = nullptr;
  const Tensor* t = optional(o, "gate");
  if (!t) return DG_GATE_NONE;
  const bool channel = t->dim() == 1 && t->size(0) == H, token = t->dim() == 2 && t->size(0) == T && t->size(1) == 1;
  if (!channel && !token)
    value_error("gate has shape " + shape_of(t->sizes()) + ", expected " + shape_of({H}) + " or " + shape_of({T, 1}));
  check(*t, "gate", {at::kFloat});
  *gate = static_cast<const float*>(t->data_ptr());
  return channel ? DG_GATE_CHANNEL : DG_GATE_TOKEN;
}

// residual_norm(R, Y, w_post, gate, alpha, w_pre, eps, values, scale mode or -1, dtype or -1)
PyObject* residual_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 10);
  need(lib.residual_norm, "dg_residual_norm");
  const Tensor& R = tensor(a[0], "R");
  const int r_code = check_values(R, "R");
  const int64_t T = R.size(0), H = R.size(1);
  if (H < 1) return failure(DG_ERR_INVALID_ARG, "dg_residual_norm");   // (its weights have no addresses)
  const Tensor* Y = optional(a[1], "Y");
  int code = small(a[9], "dtype");
  if (Y) {
    check(*Y, "Y", {at::kBFloat16, at::kFloat}, {T, H});
    if (code != -1 && code != dtype_code(*Y)) value_error("dtype is Y's where there is Y");
    code = dtype_code(*Y);
  }
  const float *w_post = weights_of(a[2], "w_post", {H}), *w_pre = weights_of(a[5], "w_pre", {H}), *gate;
  const int kind = gate_of(a[3], T, H, &gate), mode = small(a[8], "codes");
  const float alpha = real(a[4], "alpha"), eps = real(a[6], "eps");
  const bool values = truth(a[7]);
  if (!Y && (w_post || kind != DG_GATE_NONE)) value_error("w_post and gate need Y");
  if (!Y && !w_pre) value_error("without Y there must be w_pre");
  if (w_pre && !values && mode < 0) value_error("w_pre asks for values or codes");
  if (!w_pre && mode >= 0) value_error("codes need w_pre");
  Tensor Rout, N, Q, S;
  if (Y) Rout = create({T, H}, R.scalar_type(), R);
  if (w_pre && values) N = create({T, H}, code == DG_IN_BF16 ? at::kBFloat16 : at::kFloat, R);
  if (w_pre && mode >= 0) {
    Q = create({T, H}, at::kByte, R);
    S = create({T, (H + 127) / 128}, at::kFloat, R);
  }
  auto at_ = [](const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; };
  const int st = lib.residual_norm(R.data_ptr(), r_code, Y ? Y->data_ptr() : nullptr, code, w_post, gate, kind, alpha,
                                   w_pre, eps, at_(Rout), at_(N), at_(Q), static_cast<float*>(at_(S)),
                                   mode < 0 ? DG_SCALE_POW2 : mode, T, H, stream());
  if (st != DG_OK) return failure(st, "dg_residual_norm");
  return tuple(Rout, N, Q, S);
  END_HANDLE_TH_ERRORS
}

// residual_norm_bwd(dR, dN, R, Y, w_post, gate, alpha, w_pre, eps)
PyObject* residual_norm_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 9);
  need(lib.residual_norm_bwd, "dg_residual_norm_bwd");
  const Tensor *dR = optional(a[0], "dR"), *dN = optional(a[1], "dN"), *R = optional(a[2], "R"), *Y = optional(a[3], "Y");
  const bool pre = a[7] != Py_None;
  if (pre && (!R || !dN)) value_error("w_pre needs R and dN");
  if (!pre && dN) value_error("dN needs w_pre");
  if (!pre && !dR) value_error("there must be dR or dN");
  if (!pre && !Y) value_error("without Y there must be w_pre");
  const Tensor& like = pre ? *R : *dR;
  const int r_code = check_values(like, pre ? "R" : "dR");
  const int64_t T = like.size(0), H = like.size(1);
  if (H < 1) return failure(DG_ERR_INVALID_ARG, "dg_residual_norm_bwd");
  if (dR) check(*dR, "dR", {like.scalar_type()}, {T, H});
  if (R) check(*R, "R", {like.scalar_type()}, {T, H});
  if (dN) check(*dN, "dN", {at::kBFloat16, at::kFloat}, {T, H});
  if (Y) check(*Y, "Y", {at::kBFloat16, at::kFloat}, {T, H});
  if (Y && dN && Y->scalar_type() != dN->scalar_type()) value_error("Y and dN must have the same dtype");
  const int code = dtype_code(dN ? *dN : *Y);
  const float *w_post = weights_of(a[4], "w_post", {H}), *w_pre = weights_of(a[7], "w_pre", {H}), *gate;
  const int kind = gate_of(a[5], T, H, &gate);
  const float alpha = real(a[6], "alpha"), eps = real(a[8], "eps");
  if (!Y && (w_post || kind != DG_GATE_NONE)) value_error("w_post and gate need Y");
  const int64_t ws = lib.residual_norm_bwd_workspace(T, H, int(pre) + int(w_post || kind == DG_GATE_CHANNEL));
  if (ws < 0) return failure(ws, "dg_residual_norm_bwd");
  const Tensor dRout = create({T, H}, like.scalar_type(), like);
  Tensor dY, dw_post, dgate, dw_pre, work;
  if (Y) dY = create({T, H}, Y->scalar_type(), like);
  if (w_post) dw_post = create({H}, at::kFloat, like);
  if (kind != DG_GATE_NONE) dgate = create(optional(a[5], "gate")->sizes(), at::kFloat, like);
  if (w_pre) dw_pre = create({H}, at::kFloat, like);
  if (ws) work = create({ws}, at::kByte, like);
  auto in = [](const Tensor* t) -> const void* { return t ? t->data_ptr() : nullptr; };
  auto out = [](const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; };
  const int st = lib.residual_norm_bwd(in(dR), in(dN), in(pre ? R : nullptr), r_code, in(Y), code, w_post, gate, kind,
                                       alpha, w_pre, eps, out(dRout), out(dY), static_cast<float*>(out(dw_post)),
                                       static_cast<float*>(out(dgate)), static_cast<float*>(out(dw_pre)), T, H,
                                       out(work), stream());
  if (st != DG_OK) return failure(st, "dg_residual_norm_bwd");
  return tuple(dRout, dY, dw_post, dgate, dw_pre);
  END_HANDLE_TH_ERRORS
}

// A list of gradients as the arrays that the library reads.
struct Grads {
  std::vector<const void*> at;
  std::vector<int64_t> sizes;
  std::vector<int> dtypes;
  const Tensor* first = nullptr;

  Grads(PyObject* list, const char* name) : items(list) {
    if (!PyList_Check(list) && !PyTuple_Check(list)) type_error(std::string(name) + " must be a list of tensors");
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(items);
    if (n > INT32_MAX) value_error("too many tensors");
    at.reserve(n);
    sizes.reserve(n);
    dtypes.reserve(n);
    for (Py_ssize_t i = 0; i < n; ++i) {
      const Tensor& t = tensor(PySequence_Fast_GET_ITEM(items, i), name);
      check(t, name, {at::kBFloat16, at::kFloat});
      if (!first) first = &t;
      at.push_back(t.data_ptr());
      sizes.push_back(t.numel());
      dtypes.push_back(dtype_code(t));
    }
  }
  int count() const { return int(at.size()); }
  const Tensor& operator[](int i) const { return THPVariable_Unpack(PySequence_Fast_GET_ITEM(items, i)); }

 private:
  PyObject* items;       // (the caller's, which holds its tensors)
};

// grad_norm(grads)
PyObject* grad_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 1);
  need(lib.grad_norm, "dg_grad_norm");
  const Grads g(a[0], "grads");
  if (!g.first) value_error("grads must not be empty");
  const int64_t ws = lib.grad_norm_workspace(g.sizes.data(), g.dtypes.data(), g.count());
  if (ws < 0) return failure(ws, "dg_grad_norm");
  const Tensor norm = create({}, at::kFloat, *g.first);
  const Tensor work = ws ? create({ws}, at::kByte, *g.first) : Tensor();
  const int st = lib.grad_norm(g.at.data(), g.sizes.data(), g.dtypes.data(), g.count(), data<float>(norm),
                               ws ? work.data_ptr() : nullptr, stream());
  if (st != DG_OK) return failure(st, "dg_grad_norm");
  return wrap(norm);
  END_HANDLE_TH_ERRORS
}

// clip_grads(grads, norm, max_norm, out): the tensors written
PyObject* clip_grads(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arguments(n, 4);
  need(lib.clip_grads, "dg_clip_grads");
  const Grads g(a[0], "grads");
  const Tensor& norm = tensor(a[1], "norm");
  const float* at = static_cast<const float*>(scalar(norm, "norm", at::kFloat));
  const float max_norm = real(a[2], "max_norm");
  PyObject* list = a[3] == Py_None ? a[0] : a[3];
  const Grads out(list, "out");
  if (out.count() != g.count())
    value_error("out has " + std::to_string(out.count()) + " tensors, grads " + std::to_string(g.count()));
  for (int i = 0; i < g.count(); ++i)
    if (out[i].sizes() != g[i].sizes())
      value_error("out has shape " + shape_of(out[i].sizes()) + ", expected " + shape_of(g[i].sizes()));
  const int st = lib.clip_grads(g.at.data(), g.sizes.data(), g.dtypes.data(), g.count(), at, max_norm,
                                const_cast<void* const*>(out.at.data()), out.dtypes.data(), stream());
  if (st != DG_OK) return failure(st, "dg_clip_grads");
  for (int i = 0; i < out.count(); ++i)
    if (!out[i].is_inference()) out[i].unsafeGetTensorImpl()->bump_version();
  Py_INCREF(list);
  return list;
  END_HANDLE_TH_ERRORS
}

// load(path of libdg.so, DGError)
PyObject* load(PyObject*, PyObject* args) {
  const char* path;
  PyObject* error;
  if (!PyArg_ParseTuple(args, "sO", &path, &error)) return nullptr;
  void* h = dlopen(path, RTLD_NOW | RTLD_LOCAL);
  if (!h) {
    PyErr_SetString(PyExc_RuntimeError, dlerror());
    return nullptr;
  }
  bool all = true;
  auto find = [&](auto& f, const char* name) {
    f = reinterpret_cast<std::decay_t<decltype(f)>>(dlsym(h, name));
    all = all && f;
  };
  find(lib.moe_rows, "dg_moe_rows");
  find(lib.moe_sort_workspace, "dg_moe_sort_workspace");
  find(lib.moe_sort, "dg_moe_sort");
  find(lib.moe_permute, "dg_moe_permute");
  find(lib.moe_permute_fp8, "dg_moe_permute_fp8");
  find(lib.moe_combine, "dg_moe_combine");
  find(lib.moe_combine_bwd, "dg_moe_combine_bwd");
  find(lib.swiglu_fp8, "dg_swiglu_fp8");
  find(lib.swiglu_fp8_bwd, "dg_swiglu_fp8_bwd");
  find(lib.grouped_wgrad_fp8, "dg_grouped_wgrad_fp8");
  if (!all) {
    PyErr_Format(PyExc_RuntimeError, "%s lacks functions of dg.h: build it again", path);
    return nullptr;
  }
  find(lib.moe_route_workspace, "dg_moe_route_workspace");
  find(lib.moe_route, "dg_moe_route");
  find(lib.moe_route_bwd, "dg_moe_route_bwd");
  find(lib.residual_norm, "dg_residual_norm");
  find(lib.residual_norm_bwd_workspace, "dg_residual_norm_bwd_workspace");
  find(lib.residual_norm_bwd, "dg_residual_norm_bwd");
  find(lib.grad_norm_workspace, "dg_grad_norm_workspace");
  find(lib.grad_norm, "dg_grad_norm");
  find(lib.clip_grads, "dg_clip_grads");
  Py_INCREF(error);
  Py_XDECREF(dg_error);
  dg_error = error;
  Py_RETURN_NONE;
}

#define DG_FAST(NAME) {#NAME, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(NAME)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {{"load", load, METH_VARARGS, nullptr},
                         DG_FAST(moe_sort),
                         DG_FAST(moe_permute),
                         DG_FAST(moe_permute_fp8),
                         DG_FAST(moe_combine),
                         DG_FAST(moe_combine_bwd),
                         DG_FAST(swiglu_fp8),
                         DG_FAST(swiglu_fp8_bwd),
                         DG_FAST(grouped_wgrad_fp8),
                         DG_FAST(moe_route),
                         DG_FAST(moe_route_bwd),
                         DG_FAST(residual_norm),
                         DG_FAST(residual_norm_bwd),
                         DG_FAST(grad_norm),
                         DG_FAST(clip_grads),
                         {nullptr, nullptr, 0, nullptr}};
#undef DG_FAST

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_dg_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__dg_torch() { return PyModule_Create(&module); }
