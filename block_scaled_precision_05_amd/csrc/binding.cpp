// binding.cpp -- marshalling of the grouped-row operators' and the dense epilogue products'
// usual calls in native code.
//
// These operators are short (a decode step's combine runs 4 us on the GPU), and their
// Python wrappers' checks and ctypes calls take longer than that.  The functions here do
// the same marshalling for the calls that need no explanation: tensors of the right type,
// shape and layout, on the current device and its current stream.  Anything else, and a
// non-zero status, returns None and launches nothing; the Python wrapper then takes the
// call, and raises what there is to raise.  No arithmetic happens here, and the library's
// entry points are the same (their addresses come from the loaded libbsg.so).
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <stdint.h>

#include "../../include/bsg.h"

namespace {

decltype(&::sort_tokens) p_sort_tokens;
decltype(&::sort_tokens_workspace) p_sort_tokens_workspace;
decltype(&::moe_dispatch_bf16) p_moe_dispatch_bf16;
decltype(&::moe_dispatch_fp8) p_moe_dispatch_fp8;
decltype(&::moe_dispatch_fp4) p_moe_dispatch_fp4;
decltype(&::moe_combine) p_moe_combine;
decltype(&::moe_combine_backward) p_moe_combine_backward;
decltype(&::lora_add_bf16) p_lora_add_bf16;
decltype(&::lora_add_workspace) p_lora_add_workspace;
decltype(&::gemm_bf16_act) p_gemm_bf16_act;
decltype(&::gemm_fp8_act) p_gemm_fp8_act;
decltype(&::gemm_fp4_act) p_gemm_fp4_act;
decltype(&::gemm_bf16_act_backward) p_gemm_bf16_act_backward;
decltype(&::gemm_bf16_glu) p_gemm_bf16_glu;
decltype(&::gemm_bf16_glu_backward) p_gemm_bf16_glu_backward;
decltype(&::gemm_bf16_act_workspace) p_gemm_bf16_act_workspace;
decltype(&::gemm_fp8_act_workspace) p_gemm_fp8_act_workspace;
decltype(&::gemm_fp4_act_workspace) p_gemm_fp4_act_workspace;
decltype(&::gemm_bf16_act_backward_workspace) p_gemm_bf16_act_backward_workspace;
decltype(&::gemm_bf16_glu_workspace) p_gemm_bf16_glu_workspace;
decltype(&::gemm_bf16_glu_backward_workspace) p_gemm_bf16_glu_backward_workspace;
PyTypeObject* plan_type;      // the named tuple that sort_tokens returns

struct Entry {
  const char* name;
  void** slot;
};
const Entry kEntries[] = {
    {"sort_tokens", (void**)&p_sort_tokens},
    {"sort_tokens_workspace", (void**)&p_sort_tokens_workspace},
    {"moe_dispatch_bf16", (void**)&p_moe_dispatch_bf16},
    {"moe_dispatch_fp8", (void**)&p_moe_dispatch_fp8},
    {"moe_dispatch_fp4", (void**)&p_moe_dispatch_fp4},
    {"moe_combine", (void**)&p_moe_combine},
    {"moe_combine_backward", (void**)&p_moe_combine_backward},
    {"lora_add_bf16", (void**)&p_lora_add_bf16},
    {"lora_add_workspace", (void**)&p_lora_add_workspace},
    {"gemm_bf16_act", (void**)&p_gemm_bf16_act},
    {"gemm_fp8_act", (void**)&p_gemm_fp8_act},
    {"gemm_fp4_act", (void**)&p_gemm_fp4_act},
    {"gemm_bf16_act_backward", (void**)&p_gemm_bf16_act_backward},
    {"gemm_bf16_glu", (void**)&p_gemm_bf16_glu},
    {"gemm_bf16_glu_backward", (void**)&p_gemm_bf16_glu_backward},
    {"gemm_bf16_act_workspace", (void**)&p_gemm_bf16_act_workspace},
    {"gemm_fp8_act_workspace", (void**)&p_gemm_fp8_act_workspace},
    {"gemm_fp4_act_workspace", (void**)&p_gemm_fp4_act_workspace},
    {"gemm_bf16_act_backward_workspace", (void**)&p_gemm_bf16_act_backward_workspace},
    {"gemm_bf16_glu_workspace", (void**)&p_gemm_bf16_glu_workspace},
    {"gemm_bf16_glu_backward_workspace", (void**)&p_gemm_bf16_glu_backward_workspace},
};

// Allocation and launch run without the interpreter lock, as torch's own calls do.
struct NoGil {
  PyThreadState* state = PyEval_SaveThread();
  ~NoGil() { PyEval_RestoreThread(state); }
};

// A tensor argument; `ok` goes false for anything but a tensor on device `dev` with
// elements of `type`.
const at::Tensor* tensor(PyObject* o, at::ScalarType type, int64_t dev, bool& ok) {
  if (!THPVariable_Check(o)) {
    ok = false;
    return nullptr;
  }
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda() || t.get_device() != dev || t.scalar_type() != type || t.layout() != at::kStrided) ok = false;
  return &t;
}

// [rows, cols] with contiguous rows; returns the leading dimension.
int64_t matrix(const at::Tensor* t, int64_t rows, int64_t cols, bool& ok) {
  if (!ok) return 0;
  if (t->dim() != 2 || t->size(0) != rows || t->size(1) != cols || t->stride(1) != 1 || t->stride(0) < cols) {
    ok = false;
    return 0;
  }
  return t->stride(0);
}

template <class P>
P* ptr(const at::Tensor* t) {
  return t ? (P*)t->data_ptr() : nullptr;
}

// torch's allocation on the current device, which is the tensors' (at::empty without its
// trip through the dispatcher: 0.2 us of a combine's 4.7).
at::Tensor empty(at::IntArrayRef shape, at::ScalarType type) {
  return at::detail::empty_cuda(shape, type, at::Device(at::kCUDA), c10::nullopt);
}

// A tensor on part of another's storage (as_strided without its trip through the
// dispatcher: sort_tokens makes four: 6.1 -> 5.4 us a call).
at::Tensor piece(const at::Tensor& of, int64_t offset, at::IntArrayRef size, at::IntArrayRef stride) {
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(of.storage()), of.key_set(), of.dtype());
  c10::TensorImpl* const impl = t.unsafeGetTensorImpl();
  impl->set_storage_offset(offset);
  impl->set_sizes_and_strides(size, stride);
  return t;
}

struct Plan {
  const at::Tensor *offsets, *row_of, *pair_of, *row_group;
  int64_t T = 0, k = 0, rows = 0;
  Plan(PyObject* o, int64_t dev, bool& ok) {
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 4) {
      ok = false;
      return;
    }
    const at::Tensor** at_[4] = {&offsets, &row_of, &pair_of, &row_group};
    for (int i = 0; i < 4; ++i) {
      *at_[i] = tensor(PyTuple_GET_ITEM(o, i), at::kInt, dev, ok);
      if (!ok || !(*at_[i])->is_contiguous()) {
        ok = false;
        return;
      }
    }
    rows = pair_of->numel();
    if (offsets->dim() != 1 || row_of->dim() != 2 || pair_of->dim() != 1 || row_group->numel() != rows) {
      ok = false;
      return;
    }
    T = row_of->size(0);
    k = row_of->size(1);
    if (T == 0 || k == 0 || rows == 0) ok = false;      // (empty calls are not in a hurry)
  }
};

// The current device and its current stream; false where the call's first tensor is not on
// a GPU.
bool place(PyObject* first, int64_t& dev, void*& stream) {
  if (!THPVariable_Check(first) || !THPVariable_Unpack(first).is_cuda()) return false;
  const auto d = c10::hip::current_device();
  dev = d;
  stream = c10::hip::getCurrentHIPStream(d).stream();
  return true;
}

// sort_tokens(ids, G, align, cap)
PyObject* sort_tokens_(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  int64_t dev;
  void* stream;
  if (n != 4) return (PyErr_BadArgument(), nullptr);
  if (!place(a[0], dev, stream)) Py_RETURN_NONE;
  const int64_t G = PyLong_AsLongLong(a[1]), align = PyLong_AsLongLong(a[2]), cap = PyLong_AsLongLong(a[3]);
  if (PyErr_Occurred()) return nullptr;
  bool ok = G >= 1 && G <= 1024 && align >= 1 && align <= 65536 && cap >= 0 && cap <= (1 << 20);
  const at::Tensor* ids = tensor(a[0], at::kInt, dev, ok);
  if (!ok || ids->dim() != 2) Py_RETURN_NONE;
  const int64_t T = ids->size(0), k = ids->size(1), pairs = T * k;
  const int64_t ld = matrix(ids, T, k, ok);
  if (!ok || T == 0 || k == 0 || pairs > (1 << 23)) Py_RETURN_NONE;
  const int64_t heads = cap ? G : G + 1;
  const int64_t rows = cap ? G * cap : pairs + std::min(G, pairs) * (align - 1);
  at::Tensor part[4];
  int status;
  {
    NoGil g;
    // one allocation, cut into the plan's four tensors
    const at::Tensor all = empty({heads + pairs + 2 * rows}, at::kInt);
    const int64_t size[4] = {heads, pairs, rows, rows};
    int64_t off = 0;
    for (int i = 0; i < 4; ++i) {
      part[i] = i == 1 ? piece(all, off, {T, k}, {k, 1}) : piece(all, off, {size[i]}, {1});
      off += size[i];
    }
    const int64_t need = p_sort_tokens_workspace(pairs, (int32_t)G);
    at::Tensor ws;
    if (need) ws = empty({need}, at::kByte);
    status = p_sort_tokens(ids->const_data_ptr<int32_t>(), ld, T, (int32_t)k, (int32_t)G, (int32_t)align,
                           (int32_t)cap, ptr<int32_t>(&part[0]), ptr<int32_t>(&part[1]), ptr<int32_t>(&part[2]),
                           ptr<int32_t>(&part[3]), rows, need ? ws.data_ptr() : nullptr, need, stream);
  }
  if (status != BSG_OK) Py_RETURN_NONE;
  PyObject* plan = plan_type->tp_alloc(plan_type, 4);
  if (!plan) return nullptr;
  for (int i = 0; i < 4; ++i) PyTuple_SET_ITEM(plan, i, THPVariable_Wrap(std::move(part[i])));
  return plan;
  END_HANDLE_TH_ERRORS
}

// moe_dispatch_bf16(X, plan, out)
PyObject* moe_dispatch_bf16_(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  int64_t dev;
  void* stream;
  if (n != 3) return (PyErr_BadArgument(), nullptr);
  if (!place(a[0], dev, stream)) Py_RETURN_NONE;
  bool ok = true;
  const Plan p(a[1], dev, ok);
  const at::Tensor* X = tensor(a[0], at::kBFloat16, dev, ok);
  if (!ok || X->dim() != 2) Py_RETURN_NONE;
  const int64_t H = X->size(1), ldx = matrix(X, p.T, H, ok);
  const at::Tensor* out = a[2] == Py_None ? nullptr : tensor(a[2], at::kBFloat16, dev, ok);
  const int64_t ldo = out ? matrix(out, p.rows, H, ok) : H;
  if (!ok) Py_RETURN_NONE;
  at::Tensor made;
  int status;
  {
    NoGil g;
    if (!out) made = empty({p.rows, H}, at::kBFloat16);
    status = p_moe_dispatch_bf16(X->const_data_ptr(), ldx, ptr<int32_t>(p.row_of), ptr<int32_t>(p.pair_of), p.T,
                                 (int32_t)p.k, p.rows, H, out ? out->data_ptr() : made.data_ptr(), ldo, stream);
  }
  if (status != BSG_OK) Py_RETURN_NONE;
  return out ? Py_NewRef(a[2]) : THPVariable_Wrap(std::move(made));
  END_HANDLE_TH_ERRORS
}

// moe_dispatch_quantized(fp4, X, plan, rule, out, sf_out) -> (codes, scales)
PyObject* moe_dispatch_quantized_(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  int64_t dev;
  void* stream;
  if (n != 6) return (PyErr_BadArgument(), nullptr);
  if (!place(a[1], dev, stream)) Py_RETURN_NONE;
  const bool fp4 = a[0] == Py_True;
  const int64_t rule = PyLong_AsLongLong(a[3]);
  if (PyErr_Occurred()) return nullptr;
  bool ok = true;
  const Plan p(a[2], dev, ok);
  const at::Tensor* X = tensor(a[1], at::kBFloat16, dev, ok);
  if (!ok || X->dim() != 2) Py_RETURN_NONE;
  const int64_t H = X->size(1), ldx = matrix(X, p.T, H, ok);
  const int64_t gk = fp4 ? 32 : 128, cols = fp4 ? H / 2 : H, kp = (H / gk + 1) / 2;
  const at::Tensor* out = a[4] == Py_None ? nullptr : tensor(a[4], at::kByte, dev, ok);
  const at::Tensor* sf = a[5] == Py_None ? nullptr : tensor(a[5], at::kShort, dev, ok);
  const int64_t ldq = out ? matrix(out, p.rows, cols, ok) : cols;
  if (!ok || H == 0 || H % gk) Py_RETURN_NONE;
  if (sf && (sf->dim() != 2 || sf->size(1) < p.rows)) Py_RETURN_NONE;
  const int64_t ld_sf = sf ? matrix(sf, kp, sf->size(1), ok) : p.rows;
  if (!ok) Py_RETURN_NONE;
  at::Tensor q, s;
  int status;
  {
    NoGil g;
    if (!out) q = empty({p.rows, cols}, at::kByte);
    if (!sf) s = empty({kp, p.rows}, at::kShort);
    status = (fp4 ? p_moe_dispatch_fp4 : p_moe_dispatch_fp8)(
        X->const_data_ptr(), ldx, ptr<int32_t>(p.row_of), ptr<int32_t>(p.pair_of), p.T, (int32_t)p.k, p.rows, H,
        out ? out->data_ptr() : q.data_ptr(), ldq, sf ? ptr<int16_t>(sf) : ptr<int16_t>(&s), ld_sf, (int32_t)rule,
        stream);
  }
  if (status != BSG_OK) Py_RETURN_NONE;
  PyObject* r = PyTuple_New(2);
  if (!r) return nullptr;
  PyTuple_SET_ITEM(r, 0, out ? Py_NewRef(a[4]) : THPVariable_Wrap(std::move(q)));
  PyTuple_SET_ITEM(r, 1, sf ? Py_NewRef(a[5]) : THPVariable_Wrap(std::move(s)));
  return r;
  END_HANDLE_TH_ERRORS
}

// moe_combine(Y, plan, weights, out)
PyObject* moe_combine_(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  int64_t dev;
  void* stream;
  if (n != 4) return (PyErr_BadArgument(), nullptr);
  if (!place(a[0], dev, stream)) Py_RETURN_NONE;
  bool ok = true;
  const Plan p(a[1], dev, ok);
  const at::Tensor* Y = tensor(a[0], at::kBFloat16, dev, ok);
  if (!ok || Y->dim() != 2) Py_RETURN_NONE;
  const int64_t H = Y->size(1), ldy = matrix(Y, p.rows, H, ok);
  const at::Tensor* W = a[2] == Py_None ? nullptr : tensor(a[2], at::kFloat, dev, ok);
  const int64_t ldw = W ? matrix(W, p.T, p.k, ok) : p.k;
  const at::Tensor* out = a[3] == Py_None ? nullptr : tensor(a[3], at::kBFloat16, dev, ok);
  const int64_t ldo = out ? matrix(out, p.T, H, ok) : H;
  if (!ok) Py_RETURN_NONE;
  at::Tensor made;
  int status;
  {
    NoGil g;
    if (!out) made = empty({p.T, H}, at::kBFloat16);
    status = p_moe_combine(Y->const_data_ptr(), ldy, ptr<int32_t>(p.row_of), ptr<float>(W), ldw, p.T, (int32_t)p.k,
                           p.rows, H, out ? out->data_ptr() : made.data_ptr(), ldo, stream);
  }
  if (status != BSG_OK) Py_RETURN_NONE;
  return out ? Py_NewRef(a[3]) : THPVariable_Wrap(std::move(made));
  END_HANDLE_TH_ERRORS
}

// moe_combine_backward(dout, Y, plan, weights, out) -> (dY, dW)
PyObject* moe_combine_backward_(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  int64_t dev;
  void* stream;
  if (n != 5) return (PyErr_BadArgument(), nullptr);
  if (!place(a[0], dev, stream)) Py_RETURN_NONE;
  bool ok = true;
  const Plan p(a[2], dev, ok);
  const at::Tensor* dO = tensor(a[0], at::kBFloat16, dev, ok);
  const at::Tensor* Y = tensor(a[1], at::kBFloat16, dev, ok);
  if (!ok || dO->dim() != 2) Py_RETURN_NONE;
  const int64_t H = dO->size(1), ldd = matrix(dO, p.T, H, ok), ldy = matrix(Y, p.rows, H, ok);
  const at::Tensor* W = a[3] == Py_None ? nullptr : tensor(a[3], at::kFloat, dev, ok);
  const int64_t ldw = W ? matrix(W, p.T, p.k, ok) : p.k;
  const at::Tensor* out = a[4] == Py_None ? nullptr : tensor(a[4], at::kBFloat16, dev, ok);
  const int64_t ldo = out ? matrix(out, p.rows, H, ok) : H;
  if (!ok) Py_RETURN_NONE;
  at::Tensor dY, dW;
  int status;
  {
    NoGil g;
    if (!out) dY = empty({p.rows, H}, at::kBFloat16);
    dW = empty({p.T, p.k}, at::kFloat);
    status = p_moe_combine_backward(dO->const_data_ptr(), ldd, Y->const_data_ptr(), ldy, ptr<int32_t>(p.row_of),
                                    ptr<int32_t>(p.pair_of), ptr<float>(W), ldw, p.T, (int32_t)p.k, p.rows, H,
                                    out ? out->data_ptr() : dY.data_ptr(), ldo, ptr<float>(&dW), p.k, stream);
  }
  if (status != BSG_OK) Py_RETURN_NONE;
  PyObject* r = PyTuple_New(2);
  if (!r) return nullptr;
  PyTuple_SET_ITEM(r, 0, out ? Py_NewRef(a[4]) : THPVariable_Wrap(std::move(dY)));
  PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(std::move(dW)));
  return r;
  END_HANDLE_TH_ERRORS
}

// lora_add_bf16(X, A, B, plan, scale, base, out)
PyObject* lora_add_bf16_(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  int64_t dev;
  void* stream;
  if (n != 7) return (PyErr_BadArgument(), nullptr);
  if (!place(a[0], dev, stream)) Py_RETURN_NONE;
  bool ok = true;
  const Plan p(a[3], dev, ok);
  const at::Tensor* X = tensor(a[0], at::kBFloat16, dev, ok);
  const at::Tensor* A = tensor(a[1], at::kBFloat16, dev, ok);
  const at::Tensor* B = tensor(a[2], at::kBFloat16, dev, ok);
  if (!ok || p.k != 1 || A->dim() != 3 || B->dim() != 3) Py_RETURN_NONE;
  const int64_t G = A->size(0), r = A->size(1), K = A->size(2), N = B->size(1);
  const int64_t ldx = matrix(X, p.T, K, ok);
  const at::Tensor* scale = a[4] == Py_None ? nullptr : tensor(a[4], at::kFloat, dev, ok);
  const at::Tensor* base = a[5] == Py_None ? nullptr : tensor(a[5], at::kBFloat16, dev, ok);
  const at::Tensor* out = a[6] == Py_None ? nullptr : tensor(a[6], at::kBFloat16, dev, ok);
  if (!ok || G == 0 || G > 1024 || r == 0 || K == 0 || N == 0 || B->size(0) != G || B->size(2) != r ||
      A->stride(2) != 1 || B->stride(2) != 1 || p.offsets->numel() != G + 1 ||
      (scale && (scale->dim() != 1 || scale->size(0) != G || !scale->is_contiguous())))
    Py_RETURN_NONE;
  const int64_t ld_base = base ? matrix(base, p.T, N, ok) : 0, ldo = out ? matrix(out, p.T, N, ok) : N;
  if (!ok) Py_RETURN_NONE;
  at::Tensor made;
  int status;
  {
    NoGil g;
    if (!out) made = empty({p.T, N}, at::kBFloat16);
    const int64_t need = p_lora_add_workspace(p.T, p.rows, (int32_t)G, N, K, (int32_t)r);
    at::Tensor ws;
    if (need) ws = empty({need}, at::kByte);
    status = p_lora_add_bf16(X->const_data_ptr(), ldx, A->const_data_ptr(), A->stride(1), A->stride(0),
                             B->const_data_ptr(), B->stride(1), B->stride(0), ptr<float>(scale),
                             ptr<int32_t>(p.offsets), ptr<int32_t>(p.row_of), ptr<int32_t>(p.pair_of),
                             ptr<int32_t>(p.row_group), p.rows, base ? base->const_data_ptr() : nullptr, ld_base,
                             out ? out->data_ptr() : made.data_ptr(), ldo, p.T, (int32_t)G, N, K, (int32_t)r,
                             need ? ws.data_ptr() : nullptr, need, stream);
  }
  if (status != BSG_OK) Py_RETURN_NONE;
  return out ? Py_NewRef(a[6]) : THPVariable_Wrap(std::move(made));
  END_HANDLE_TH_ERRORS
}

// Scratch memory of a call, freed (to torch's allocator, on the stream) when it returns.
struct Scratch {
  at::Tensor t;
  void* p = nullptr;
  int64_t bytes;
  explicit Scratch(int64_t need) : bytes(need) {
    if (need) {
      t = empty({need}, at::kByte);
      p = t.data_ptr();
    }
  }
};

// bias [N], residual [M, N] and output [M, N] of an act call.
struct Epilogue {
  const at::Tensor *bias, *R, *out;
  int64_t ldr, ldd;
  Epilogue(PyObject* bias_, PyObject* R_, PyObject* out_, int64_t M, int64_t N, int64_t dev, bool& ok) {
    bias = bias_ == Py_None ? nullptr : tensor(bias_, at::kBFloat16, dev, ok);
    R = R_ == Py_None ? nullptr : tensor(R_, at::kBFloat16, dev, ok);
    out = out_ == Py_None ? nullptr : tensor(out_, at::kBFloat16, dev, ok);
    if (ok && bias && (bias->dim() != 1 || bias->size(0) != N || !bias->is_contiguous())) ok = false;
    ldr = R ? matrix(R, M, N, ok) : 0;
    ldd = out ? matrix(out, M, N, ok) : N;
  }
};

// gemm_bf16_act(A, B, bias, act, residual, out, preact)
PyObject* gemm_bf16_act_(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  int64_t dev;
  void* stream;
  if (n != 7) return (PyErr_BadArgument(), nullptr);
  if (!place(a[0], dev, stream)) Py_RETURN_NONE;
  const int64_t act = PyLong_AsLongLong(a[3]);
  if (PyErr_Occurred()) return nullptr;
  bool ok = true;
  const at::Tensor* A = tensor(a[0], at::kBFloat16, dev, ok);
  const at::Tensor* B = tensor(a[1], at::kBFloat16, dev, ok);
  if (!ok || A->dim() != 2 || B->dim() != 2) Py_RETURN_NONE;
  const int64_t M = A->size(0), K = A->size(1), N = B->size(0);
  const int64_t lda = matrix(A, M, K, ok), ldb = matrix(B, N, K, ok);
  const Epilogue e(a[2], a[4], a[5], M, N, dev, ok);
  const at::Tensor* Z = a[6] == Py_None ? nullptr : tensor(a[6], at::kBFloat16, dev, ok);
  const int64_t ldz = Z ? matrix(Z, M, N, ok) : 0;
  if (!ok || M == 0 || N == 0 || K == 0) Py_RETURN_NONE;
  at::Tensor made;
  int status;
  {
    NoGil g;
    if (!e.out) made = empty({M, N}, at::kBFloat16);
    const Scratch ws(p_gemm_bf16_act_workspace(M, N, K));
    status = p_gemm_bf16_act(A->const_data_ptr(), lda, B->const_data_ptr(), ldb, ptr<void>(e.bias), (int32_t)act,
                             ptr<void>(e.R), e.ldr, e.out ? e.out->data_ptr() : made.data_ptr(), e.ldd, ptr<void>(Z),
                             ldz, M, N, K, ws.p, ws.bytes, stream);
  }
  if (status != BSG_OK) Py_RETURN_NONE;
  return e.out ? Py_NewRef(a[5]) : THPVariable_Wrap(std::move(made));
  END_HANDLE_TH_ERRORS
}

// A tensor of codes: bytes, or e4m3 values.
const at::Tensor* codes(PyObject* o, bool fp4, int64_t dev, bool& ok) {
  if (!THPVariable_Check(o)) {
    ok = false;
    return nullptr;
  }
  const at::ScalarType t = THPVariable_Unpack(o).scalar_type();
  return tensor(o, !fp4 && t == at::kFloat8_e4m3fn ? t : at::kByte, dev, ok);
}

// gemm_scaled_act(fp4, A, sfa, B, sfb, sfb_gran_mn, bias, act, residual, out)
PyObject* gemm_scaled_act_(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  int64_t dev;
  void* stream;
  if (n != 10) return (PyErr_BadArgument(), nullptr);
  if (!place(a[1], dev, stream)) Py_RETURN_NONE;
  const bool fp4 = a[0] == Py_True;
  const int64_t gran = PyLong_AsLongLong(a[5]), act = PyLong_AsLongLong(a[7]);
  if (PyErr_Occurred()) return nullptr;
  bool ok = gran == 1 || gran == 128;
  const at::Tensor* A = codes(a[1], fp4, dev, ok);
  const at::Tensor* B = codes(a[3], fp4, dev, ok);
  const at::Tensor* sfa = tensor(a[2], at::kShort, dev, ok);
  const at::Tensor* sfb = tensor(a[4], at::kShort, dev, ok);
  if (!ok || A->dim() != 2 || B->dim() != 2 || sfa->dim() != 2 || sfb->dim() != 2) Py_RETURN_NONE;
  const int64_t M = A->size(0), bytes = A->size(1), N = B->size(0), K = fp4 ? 2 * bytes : bytes, gk = fp4 ? 32 : 128;
  const int64_t lda = matrix(A, M, bytes, ok), ldb = matrix(B, N, bytes, ok);
  const int64_t kp = (K / gk + 1) / 2, rows_b = (N + gran - 1) / gran;
  if (sfa->size(1) < M || sfb->size(1) < rows_b) ok = false;
  const int64_t ld_sfa = matrix(sfa, kp, sfa->size(1), ok), ld_sfb = matrix(sfb, kp, sfb->size(1), ok);
  const Epilogue e(a[6], a[8], a[9], M, N, dev, ok);
  if (!ok || M == 0 || N == 0 || K == 0) Py_RETURN_NONE;
  at::Tensor made;
  int status;
  {
    NoGil g;
    if (!e.out) made = empty({M, N}, at::kBFloat16);
    void* const D = e.out ? e.out->data_ptr() : made.data_ptr();
    const Scratch ws((fp4 ? p_gemm_fp4_act_workspace : p_gemm_fp8_act_workspace)(M, N, K));
    status = fp4 ? p_gemm_fp4_act(A->const_data_ptr(), lda, ptr<int16_t>(sfa), ld_sfa, B->const_data_ptr(), ldb,
                                  ptr<int16_t>(sfb), ld_sfb, ptr<void>(e.bias), (int32_t)act, ptr<void>(e.R), e.ldr, D,
                                  e.ldd, M, N, K, ws.p, ws.bytes, stream)
                 : p_gemm_fp8_act(A->const_data_ptr(), lda, ptr<int16_t>(sfa), ld_sfa, B->const_data_ptr(), ldb,
                                  ptr<int16_t>(sfb), ld_sfb, (int32_t)gran, ptr<void>(e.bias), (int32_t)act,
                                  ptr<void>(e.R), e.ldr, D, e.ldd, M, N, K, ws.p, ws.bytes, stream);
  }
  if (status != BSG_OK) Py_RETURN_NONE;
  return e.out ? Py_NewRef(a[9]) : THPVariable_Wrap(std::move(made));
  END_HANDLE_TH_ERRORS
}

// The result tuple of a backward call: what was not asked for is None.
PyObject* results(at::Tensor* t, int count) {
  PyObject* r = PyTuple_New(count);
  if (!r) return nullptr;
  for (int i = 0; i < count; ++i)
    PyTuple_SET_ITEM(r, i, t[i].defined() ? THPVariable_Wrap(std::move(t[i])) : Py_NewRef(Py_None));
  return r;
}

// gemm_bf16_act_backward(dout, A, B, preact, act, need_a, need_b, need_bias) -> (dA, dB, dbias)
PyObject* gemm_bf16_act_backward_(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  int64_t dev;
  void* stream;
  if (n != 8) return (PyErr_BadArgument(), nullptr);
  if (!place(a[0], dev, stream)) Py_RETURN_NONE;
  const int64_t act = PyLong_AsLongLong(a[4]);
  if (PyErr_Occurred()) return nullptr;
  bool need[3];
  for (int i = 0; i < 3; ++i) {
    const int v = PyObject_IsTrue(a[5 + i]);
    if (v < 0) return nullptr;
    need[i] = v;
  }
  bool ok = true;
  const at::Tensor* dO = tensor(a[0], at::kBFloat16, dev, ok);
  const at::Tensor* A = tensor(a[1], at::kBFloat16, dev, ok);
  const at::Tensor* B = tensor(a[2], at::kBFloat16, dev, ok);
  const at::Tensor* Z = a[3] == Py_None ? nullptr : tensor(a[3], at::kBFloat16, dev, ok);
  if (!ok || A->dim() != 2 || B->dim() != 2 || (!Z && act != 0)) Py_RETURN_NONE;
  const int64_t M = A->size(0), K = A->size(1), N = B->size(0);
  const int64_t lda = matrix(A, M, K, ok), ldb = matrix(B, N, K, ok), ldd = matrix(dO, M, N, ok);
  const int64_t ldz = Z ? matrix(Z, M, N, ok) : 0;
  if (!ok || M == 0 || N == 0 || K == 0) Py_RETURN_NONE;
  at::Tensor out[3];
  int status;
  {
    NoGil g;
    if (need[0]) out[0] = empty({M, K}, at::kBFloat16);
    if (need[1]) out[1] = empty({N, K}, at::kBFloat16);
    if (need[2]) out[2] = empty({N}, at::kFloat);
    const Scratch ws(p_gemm_bf16_act_backward_workspace(M, N, K));
    status = p_gemm_bf16_act_backward(dO->const_data_ptr(), ldd, ptr<void>(Z), ldz, A->const_data_ptr(), lda,
                                      B->const_data_ptr(), ldb, (int32_t)act, need[0] ? out[0].data_ptr() : nullptr, K,
                                      need[1] ? out[1].data_ptr() : nullptr, K,
                                      need[2] ? ptr<float>(&out[2]) : nullptr, M, N, K, ws.p, ws.bytes, stream);
  }
  if (status != BSG_OK) Py_RETURN_NONE;
  return results(out, 3);
  END_HANDLE_TH_ERRORS
}

// gemm_bf16_glu(X, W13, act, out, preact)
PyObject* gemm_bf16_glu_(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  int64_t dev;
  void* stream;
  if (n != 5) return (PyErr_BadArgument(), nullptr);
  if (!place(a[0], dev, stream)) Py_RETURN_NONE;
  const int64_t act = PyLong_AsLongLong(a[2]);
  if (PyErr_Occurred()) return nullptr;
  bool ok = true;
  const at::Tensor* X = tensor(a[0], at::kBFloat16, dev, ok);
  const at::Tensor* W = tensor(a[1], at::kBFloat16, dev, ok);
  const at::Tensor* out = a[3] == Py_None ? nullptr : tensor(a[3], at::kBFloat16, dev, ok);
  const at::Tensor* Z = a[4] == Py_None ? nullptr : tensor(a[4], at::kBFloat16, dev, ok);
  if (!ok || X->dim() != 2 || W->dim() != 2 || W->size(0) % 2) Py_RETURN_NONE;
  const int64_t M = X->size(0), K = X->size(1), inter = W->size(0) / 2;
  const int64_t ldx = matrix(X, M, K, ok), ldw = matrix(W, 2 * inter, K, ok);
  const int64_t ldh = out ? matrix(out, M, inter, ok) : inter, ldz = Z ? matrix(Z, M, 2 * inter, ok) : 0;
  if (!ok || M == 0 || inter == 0 || K == 0) Py_RETURN_NONE;
  at::Tensor made;
  int status;
  {
    NoGil g;
    if (!out) made = empty({M, inter}, at::kBFloat16);
    const Scratch ws(p_gemm_bf16_glu_workspace(M, inter, K));
    status = p_gemm_bf16_glu(X->const_data_ptr(), ldx, W->const_data_ptr(), ldw, (int32_t)act,
                             out ? out->data_ptr() : made.data_ptr(), ldh, ptr<void>(Z), ldz, M, inter, K, ws.p,
                             ws.bytes, stream);
  }
  if (status != BSG_OK) Py_RETURN_NONE;
  return out ? Py_NewRef(a[3]) : THPVariable_Wrap(std::move(made));
  END_HANDLE_TH_ERRORS
}

// gemm_bf16_glu_backward(dout, X, W13, preact, act, need_x, need_w) -> (dX, dW13)
PyObject* gemm_bf16_glu_backward_(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  int64_t dev;
  void* stream;
  if (n != 7) return (PyErr_BadArgument(), nullptr);
  if (!place(a[0], dev, stream)) Py_RETURN_NONE;
  const int64_t act = PyLong_AsLongLong(a[4]);
  if (PyErr_Occurred()) return nullptr;
  const int need_x = PyObject_IsTrue(a[5]), need_w = PyObject_IsTrue(a[6]);
  if (need_x < 0 || need_w < 0) return nullptr;
  bool ok = true;
  const at::Tensor* dO = tensor(a[0], at::kBFloat16, dev, ok);
  const at::Tensor* X = tensor(a[1], at::kBFloat16, dev, ok);
  const at::Tensor* W = tensor(a[2], at::kBFloat16, dev, ok);
  const at::Tensor* Z = tensor(a[3], at::kBFloat16, dev, ok);
  if (!ok || X->dim() != 2 || W->dim() != 2 || W->size(0) % 2) Py_RETURN_NONE;
  const int64_t M = X->size(0), K = X->size(1), inter = W->size(0) / 2;
  const int64_t ldx = matrix(X, M, K, ok), ldw = matrix(W, 2 * inter, K, ok), ldd = matrix(dO, M, inter, ok);
  const int64_t ldz = matrix(Z, M, 2 * inter, ok);
  if (!ok || M == 0 || inter == 0 || K == 0) Py_RETURN_NONE;
  at::Tensor out[2];
  int status;
  {
    NoGil g;
    if (need_x) out[0] = empty({M, K}, at::kBFloat16);
    if (need_w) out[1] = empty({2 * inter, K}, at::kBFloat16);
    const Scratch ws(p_gemm_bf16_glu_backward_workspace(M, inter, K));
    status = p_gemm_bf16_glu_backward(dO->const_data_ptr(), ldd, Z->const_data_ptr(), ldz, X->const_data_ptr(), ldx,
                                      W->const_data_ptr(), ldw, (int32_t)act, need_x ? out[0].data_ptr() : nullptr, K,
                                      need_w ? out[1].data_ptr() : nullptr, K, M, inter, K, ws.p, ws.bytes, stream);
  }
  if (status != BSG_OK) Py_RETURN_NONE;
  return results(out, 2);
  END_HANDLE_TH_ERRORS
}

// init(plan_type, {name: address of the library's entry point})
PyObject* init_(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 2 || !PyType_Check(a[0]) || !PyType_IsSubtype((PyTypeObject*)a[0], &PyTuple_Type) || !PyDict_Check(a[1])) {
    PyErr_BadArgument();
    return nullptr;
  }
  for (const Entry& e : kEntries) {
    PyObject* v = PyDict_GetItemString(a[1], e.name);
    if (!v) {
      PyErr_SetString(PyExc_KeyError, e.name);
      return nullptr;
    }
    *e.slot = PyLong_AsVoidPtr(v);
    if (PyErr_Occurred()) return nullptr;
  }
  Py_INCREF(a[0]);
  plan_type = (PyTypeObject*)a[0];
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"init", (PyCFunction)(void (*)(void))init_, METH_FASTCALL, nullptr},
    {"sort_tokens", (PyCFunction)(void (*)(void))sort_tokens_, METH_FASTCALL, nullptr},
    {"moe_dispatch_bf16", (PyCFunction)(void (*)(void))moe_dispatch_bf16_, METH_FASTCALL, nullptr},
    {"moe_dispatch_quantized", (PyCFunction)(void (*)(void))moe_dispatch_quantized_, METH_FASTCALL, nullptr},
    {"moe_combine", (PyCFunction)(void (*)(void))moe_combine_, METH_FASTCALL, nullptr},
    {"moe_combine_backward", (PyCFunction)(void (*)(void))moe_combine_backward_, METH_FASTCALL, nullptr},
    {"lora_add_bf16", (PyCFunction)(void (*)(void))lora_add_bf16_, METH_FASTCALL, nullptr},
    {"gemm_bf16_act", (PyCFunction)(void (*)(void))gemm_bf16_act_, METH_FASTCALL, nullptr},
    {"gemm_scaled_act", (PyCFunction)(void (*)(void))gemm_scaled_act_, METH_FASTCALL, nullptr},
    {"gemm_bf16_act_backward", (PyCFunction)(void (*)(void))gemm_bf16_act_backward_, METH_FASTCALL, nullptr},
    {"gemm_bf16_glu", (PyCFunction)(void (*)(void))gemm_bf16_glu_, METH_FASTCALL, nullptr},
    {"gemm_bf16_glu_backward", (PyCFunction)(void (*)(void))gemm_bf16_glu_backward_, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", "Marshalling of the grouped-row operators and the dense epilogue products.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
