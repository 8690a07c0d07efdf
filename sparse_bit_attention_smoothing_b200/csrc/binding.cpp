// binding.cpp -- the Python entry points of the operators around the
// attention: checks of the tensors, allocation of outputs and workspaces, and
// the call of the C ABI.  They serve single tokens too, whose kernels take a
// few microseconds, so this layer is compiled (18 us a call in Python, 6 here).
// Work runs on the current stream of the tensors' device.
#include <ATen/ATen.h>
#include <ATen/core/grad_mode.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/extension.h>

#include <array>
#include <optional>

#include "../../include/sagesla.h"

namespace py = pybind11;
using at::Tensor;
using MaybeTensor = std::optional<Tensor>;

namespace {

#define NEED(ok, ...) TORCH_CHECK_VALUE(ok, __VA_ARGS__)

void check(int rc, const char* where) {
  if (rc == SAGESLA_OK) return;
  py::object type = py::module_::import("sparse_bit_attention_smoothing_b200").attr("SageSLAError");
  py::object e = type(rc, where);
  PyErr_SetObject(type.ptr(), e.ptr());
  throw py::error_already_set();
}

int type_code(const Tensor& t, bool fp32 = false) {
  const auto s = t.scalar_type();
  if (s == at::kBFloat16) return SAGESLA_BF16;
  if (s == at::kHalf) return SAGESLA_FP16;
  if (fp32 && s == at::kFloat) return SAGESLA_FP32;
  NEED(false, t.scalar_type(), " is not supported (bfloat16, float16", fp32 ? ", float32)" : ")");
  return -1;
}

void same_device(const Tensor& first, std::initializer_list<const Tensor*> others) {
  NEED(first.is_cuda(), "CUDA tensors are needed");
  for (const Tensor* t : others) NEED(!t || t->device() == first.device(), "the tensors are on different devices");
}
// The call works outside autograd.  Where a gradient would be wanted of an
// argument, the results would be cut from its graph without a word.
void no_gradient(std::initializer_list<const Tensor*> ts, const char* where) {
  if (!at::GradMode::is_enabled()) return;
  for (const Tensor* t : ts)
    NEED(!t || !t->requires_grad(), where,
         " records no gradient and an argument requires one: call it under torch.no_grad() or in a torch.autograd.Function "
         "(sagesla_qk_norm_rope_bwd is the backward pass)");
}
const Tensor* opt(const MaybeTensor& t) { return t ? &*t : nullptr; }
void* ptr(const Tensor& t) { return t.data_ptr(); }
void* ptr(const MaybeTensor& t) { return t ? t->data_ptr() : nullptr; }

// The tensors' device and its current stream, for the length of a call.
struct Here {
  c10::cuda::CUDAGuard guard;
  sagesla_stream_t st;
  explicit Here(const Tensor& t)
      : guard(t.device()), st(c10::cuda::getCurrentCUDAStream(t.device().index()).stream()) {}
};

int small(int64_t v, const char* what) {
  NEED(v <= INT32_MAX, what, " is too large");
  return (int)v;
}

void vector(const Tensor& t, int64_t n, at::ScalarType type, const char* what) {
  NEED(t.scalar_type() == type && t.dim() == 1 && t.size(0) == n && t.is_contiguous(), what, " must be a contiguous ", type,
       " vector of ", n);
}

// Both on the current stream of the current device, from torch's allocator and
// past its dispatcher (two outputs: 6.1 -> 5.8 us a call, one and a workspace: 7.6 -> 7.3).
Tensor make(at::IntArrayRef shape, at::ScalarType type, const Tensor& like) {
  return at::detail::empty_cuda(shape, type, like.device(), std::nullopt);
}
c10::DataPtr scratch(int64_t bytes) { return c10::cuda::CUDACachingAllocator::get()->allocate((size_t)bytes); }

// ------------------------------------------------- W8A8, per token/channel
py::tuple w8a8_token_quant(const Tensor& a) {
  NEED(a.dim() == 2 && (a.size(1) <= 1 || a.stride(1) == 1), "a must be a matrix with contiguous rows");
  const int dt = type_code(a);
  same_device(a, {});
  Here here(a);
  Tensor codes = make({a.size(0), a.size(1)}, at::kChar, a), scales = make({a.size(0)}, at::kFloat, a);
  check(sagesla_w8a8_token_quant(ptr(a), dt, small(a.size(0), "rows"), small(a.size(1), "cols"), a.stride(0),
                                 (int8_t*)ptr(codes), (float*)ptr(scales), here.st),
        "sagesla_w8a8_token_quant");
  return py::make_tuple(codes, scales);
}

int64_t token_weight(const Tensor& wq, const Tensor& sw, const MaybeTensor& bias, int64_t K, at::ScalarType type) {
  NEED(wq.dim() == 2 && wq.scalar_type() == at::kChar && wq.is_contiguous() && wq.size(1) == K,
       "wq must be a contiguous int8 [N, ", K, "] matrix");
  vector(sw, wq.size(0), at::kFloat, "sw");
  if (bias) vector(*bias, wq.size(0), type, "bias");
  return wq.size(0);
}

Tensor token_out(const MaybeTensor& y, int64_t M, int64_t N, at::ScalarType type, const Tensor& like) {
  if (!y) return make({M, N}, type, like);
  NEED(y->dim() == 2 && y->size(0) == M && y->size(1) == N && y->scalar_type() == type && y->is_contiguous(),
       "y must be a contiguous ", type, " [", M, ", ", N, "]");
  return *y;
}

Tensor w8a8_token_gemm(const Tensor& xq, const Tensor& sx, const Tensor& wq, const Tensor& sw, const MaybeTensor& bias,
                       std::optional<at::ScalarType> dtype, const MaybeTensor& y) {
  const at::ScalarType type = dtype ? *dtype : y ? y->scalar_type() : at::kBFloat16;
  NEED(xq.dim() == 2 && xq.scalar_type() == at::kChar && xq.is_contiguous(),
       "xq must be a contiguous int8 [M, K] matrix");
  const int64_t M = xq.size(0), K = xq.size(1);
  vector(sx, M, at::kFloat, "sx");
  const int64_t N = token_weight(wq, sw, bias, K, type);
  same_device(xq, {&sx, &wq, &sw, opt(bias), opt(y)});
  Here here(xq);
  Tensor out = token_out(y, M, N, type, xq);
  check(sagesla_w8a8_token_gemm((const int8_t*)ptr(xq), (const float*)ptr(sx), (const int8_t*)ptr(wq),
                                (const float*)ptr(sw), ptr(bias), ptr(out), type_code(out), small(M, "M"),
                                small(N, "N"), small(K, "K"), here.st),
        "sagesla_w8a8_token_gemm");
  return out;
}

Tensor w8a8_token_linear(const Tensor& x, const Tensor& wq, const Tensor& sw, const MaybeTensor& bias,
                         const MaybeTensor& y) {
  NEED(x.dim() == 2 && (x.size(1) <= 1 || x.stride(1) == 1), "x must be a matrix with contiguous rows");
  const int dt = type_code(x);
  const int64_t M = x.size(0), K = x.size(1), N = token_weight(wq, sw, bias, K, x.scalar_type());
  same_device(x, {&wq, &sw, opt(bias), opt(y)});
  Here here(x);
  Tensor out = token_out(y, M, N, x.scalar_type(), x);
  long long bytes = 0;
  check(sagesla_w8a8_token_workspace(small(M, "M"), small(K, "K"), &bytes), "sagesla_w8a8_token_linear");
  const c10::DataPtr ws = scratch(bytes);
  check(sagesla_w8a8_token_linear(ptr(x), x.stride(0), (const int8_t*)ptr(wq), (const float*)ptr(sw), ptr(bias),
                                  ptr(out), dt, (int)M, small(N, "N"), (int)K, ws.get(), bytes, here.st),
        "sagesla_w8a8_token_linear");
  return out;
}

// -------------------------------------------------------- rows of channels
int64_t rows4(const Tensor& t, int64_t B, int64_t N, int64_t d, at::ScalarType type, const char* what) {
  NEED(t.dim() == 4 && t.size(0) == B && t.size(1) == N && t.size(3) == d && t.scalar_type() == type &&
           t.stride(3) == 1,
       what, " must be a ", type, " [", B, ", ", N, ", heads, ", d, "] tensor with contiguous channels");
  return t.size(2);
}

Tensor rows_out(const MaybeTensor& t, int64_t B, int64_t N, int64_t H, int64_t d, const Tensor& like, bool head_major,
                const char* what) {
  if (t) {
    NEED(rows4(*t, B, N, d, like.scalar_type(), what) == H, what, " must have ", H, " heads");
    return *t;
  }
  if (head_major) return make({B, H, N, d}, like.scalar_type(), like).transpose(1, 2);
  return make({B, N, H, d}, like.scalar_type(), like);
}

template <size_t n>
std::array<int64_t, 3 * n> strides(const std::array<const Tensor*, n>& ts) {
  std::array<int64_t, 3 * n> s{};
  for (size_t i = 0; i < n; ++i)
    if (ts[i])
      for (int j = 0; j < 3; ++j) s[3 * i + j] = ts[i]->stride(j);
  return s;
}

struct RopeShape {
  int B, N, Hq, Hk, d, rot, T, dt;
};
RopeShape rope_shape(const Tensor& q, const MaybeTensor& k, const Tensor& gq, const MaybeTensor& gk, const Tensor& cos,
                     const Tensor& sin, const MaybeTensor& pos) {
  NEED(q.dim() == 4 && q.stride(3) == 1, "q must be a [B, N, H, d] tensor with contiguous channels");
  RopeShape r;
  const auto type = q.scalar_type();
  r.dt = type_code(q, true);
  const int64_t B = q.size(0), N = q.size(1), d = q.size(3);
  r.B = small(B, "B"), r.N = small(N, "N"), r.Hq = small(q.size(2), "H"), r.d = small(d, "d");
  r.Hk = k ? small(rows4(*k, B, N, d, type, "k"), "H") : 0;
  vector(gq, d, type, "gamma_q");
  if (k) {
    NEED(gk.has_value(), "k needs gamma_k");
    vector(*gk, d, type, "gamma_k");
  }
  NEED(cos.dim() == 2 && cos.sizes() == sin.sizes() && cos.scalar_type() == at::kFloat &&
           sin.scalar_type() == at::kFloat && cos.is_contiguous() && sin.is_contiguous(),
       "cos and sin must be contiguous fp32 [T, rot/2] tables");
  r.T = small(cos.size(0), "T"), r.rot = small(2 * cos.size(1), "rot");
  NEED(!pos || (pos->scalar_type() == at::kInt && pos->dim() == 2 && pos->size(0) == B && pos->size(1) == N &&
                pos->is_contiguous()),
       "pos must be a contiguous int32 [", B, ", ", N, "] tensor");
  return r;
}

py::tuple qk_norm_rope(const Tensor& q, const MaybeTensor& k, const Tensor& gq, const MaybeTensor& gk,
                       const Tensor& cos, const Tensor& sin, const MaybeTensor& pos, double eps, bool interleaved,
                       const MaybeTensor& q_out, const MaybeTensor& k_out, bool head_major) {
  no_gradient({&q, opt(k), &gq, k ? opt(gk) : nullptr, &cos, &sin}, "sagesla_qk_norm_rope");
  const RopeShape r = rope_shape(q, k, gq, gk, cos, sin, pos);
  same_device(q, {opt(k), &gq, opt(gk), &cos, &sin, opt(pos), opt(q_out), opt(k_out)});
  Here here(q);
  Tensor qo = rows_out(q_out, r.B, r.N, r.Hq, r.d, q, head_major, "q_out");
  MaybeTensor ko;
  if (k) ko = rows_out(k_out, r.B, r.N, r.Hk, r.d, q, head_major, "k_out");
  const auto s = strides<4>({&q, opt(k), &qo, opt(ko)});
  check(sagesla_qk_norm_rope(ptr(q), ptr(k), ptr(gq), k ? ptr(gk) : nullptr, (float)eps, (const float*)ptr(cos),
                             (const float*)ptr(sin), (const int32_t*)ptr(pos), ptr(qo), ptr(ko), r.dt, r.B, r.N, r.Hq,
                             r.Hk, r.d, r.rot, r.T, interleaved, s.data(), here.st),
        "sagesla_qk_norm_rope");
  if (head_major) {
    qo = qo.transpose(1, 2);
    if (ko) ko = ko->transpose(1, 2);
  }
  return py::make_tuple(qo, ko);
}

py::tuple qk_norm_rope_bwd(const Tensor& dq_out, const MaybeTensor& dk_out, const Tensor& q, const MaybeTensor& k,
                           const Tensor& gq, const MaybeTensor& gk, const Tensor& cos, const Tensor& sin,
                           const MaybeTensor& pos, double eps, bool interleaved, const MaybeTensor& dq,
                           const MaybeTensor& dk) {
  no_gradient({&dq_out, k ? opt(dk_out) : nullptr, &q, opt(k), &gq, k ? opt(gk) : nullptr, &cos, &sin}, "sagesla_qk_norm_rope_bwd");
  const RopeShape r = rope_shape(q, k, gq, gk, cos, sin, pos);
  const auto type = q.scalar_type();
  NEED(rows4(dq_out, r.B, r.N, r.d, type, "dq_out") == r.Hq, "dq_out must have ", r.Hq, " heads");
  NEED(!k || (dk_out && rows4(*dk_out, r.B, r.N, r.d, type, "dk_out") == r.Hk), "dk_out must have ", r.Hk, " heads");
  same_device(q, {&dq_out, opt(dk_out), opt(k), &gq, opt(gk), &cos, &sin, opt(pos), opt(dq), opt(dk)});
  Here here(q);
  Tensor oq = rows_out(dq, r.B, r.N, r.Hq, r.d, q, false, "dq");
  MaybeTensor ok;
  if (k) ok = rows_out(dk, r.B, r.N, r.Hk, r.d, q, false, "dk");
  Tensor dg = make({2, r.d}, at::kFloat, q);
  long long bytes = 0;
  check(sagesla_qk_norm_rope_bwd_workspace(r.B, r.N, r.Hq, r.Hk, r.d, &bytes), "sagesla_qk_norm_rope_bwd");
  const c10::DataPtr ws = scratch(bytes);
  float* g = (float*)ptr(dg);
  const auto s = strides<6>({&dq_out, k ? opt(dk_out) : nullptr, &q, opt(k), &oq, opt(ok)});
  check(sagesla_qk_norm_rope_bwd(ptr(dq_out), k ? ptr(dk_out) : nullptr, ptr(q), ptr(k), ptr(gq), k ? ptr(gk) : nullptr,
                                 (float)eps, (const float*)ptr(cos), (const float*)ptr(sin), (const int32_t*)ptr(pos),
                                 ptr(oq), ptr(ok), g, k ? g + r.d : nullptr, r.dt, r.B, r.N, r.Hq, r.Hk, r.d, r.rot,
                                 r.T, interleaved, s.data(), ws.get(), bytes, here.st),
        "sagesla_qk_norm_rope_bwd");
  MaybeTensor gk_out;
  if (k) gk_out = dg[1];
  return py::make_tuple(oq, ok, dg[0], gk_out);
}

// ------------------------------------------- linear attention with a decay
void decay_state(const MaybeTensor& t, int64_t B, int64_t H, int64_t d, const char* what) {
  if (!t) return;
  NEED(t->scalar_type() == at::kFloat && t->dim() == 4 && t->size(0) == B && t->size(1) == H && t->size(2) == d &&
           t->size(3) == d && t->is_contiguous(),
       what, " must be a contiguous fp32 [", B, ", ", H, ", ", d, ", ", d, "] tensor");
}

py::tuple linear_decay(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& log_decay,
                       const MaybeTensor& state, const MaybeTensor& lens, double scale, const MaybeTensor& out,
                       const MaybeTensor& state_out, bool head_major) {
  NEED(q.dim() == 4 && q.scalar_type() == at::kBFloat16, "q must be a bf16 [B, N, H, d] tensor");
  const int64_t B = q.size(0), N = q.size(1), H = q.size(2), d = q.size(3);
  rows4(q, B, N, d, at::kBFloat16, "q");
  const int64_t Hk = rows4(k, B, N, d, at::kBFloat16, "k");
  NEED(rows4(v, B, N, d, at::kBFloat16, "v") == Hk, "k and v must have the same heads");
  vector(log_decay, H, at::kFloat, "log_decay");
  decay_state(state, B, H, d, "state");
  decay_state(state_out, B, H, d, "state_out");
  if (lens) vector(*lens, B, at::kInt, "lens");
  same_device(q, {&k, &v, &log_decay, opt(state), opt(lens), opt(out), opt(state_out)});
  Here here(q);
  Tensor o = rows_out(out, B, N, H, d, q, head_major, "out");
  Tensor so = state_out ? *state_out : make({B, H, d, d}, at::kFloat, q);
  long long bytes = 0;
  check(sagesla_linear_decay_workspace(small(B, "B"), small(N, "N"), small(H, "H"), small(d, "d"), &bytes),
        "sagesla_linear_decay");
  c10::DataPtr ws;
  if (bytes) ws = scratch(bytes);
  const auto s = strides<4>({&q, &k, &v, &o});
  check(sagesla_linear_decay(ptr(q), ptr(k), ptr(v), (const float*)ptr(log_decay), (const float*)ptr(state),
                             (const int32_t*)ptr(lens), (float)scale, ptr(o), (float*)ptr(so), (int)B, (int)N, (int)H,
                             small(Hk, "H"), (int)d, s.data(), ws.get(), bytes, here.st),
        "sagesla_linear_decay");
  return py::make_tuple(head_major ? o.transpose(1, 2) : o, so);
}

py::tuple linear_decay_step(const Tensor& q, const Tensor& k, const Tensor& v, const Tensor& log_decay,
                            const Tensor& state, double scale, const MaybeTensor& out, const MaybeTensor& state_out) {
  const auto row = [](const Tensor& t, int64_t B, int64_t H, int64_t d, const char* what) {
    NEED(t.dim() == 3 && t.scalar_type() == at::kBFloat16 && t.size(0) == B && t.size(1) == H && t.size(2) == d &&
             t.stride(2) == 1,
         what, " must be a bf16 [", B, ", ", H, ", ", d, "] tensor with contiguous channels");
  };
  NEED(q.dim() == 3 && k.dim() == 3, "q and k must be [B, heads, d] tensors");
  const int64_t B = q.size(0), H = q.size(1), d = q.size(2), Hk = k.size(1);
  row(q, B, H, d, "q");
  row(k, B, Hk, d, "k");
  row(v, B, Hk, d, "v");
  vector(log_decay, H, at::kFloat, "log_decay");
  decay_state(state, B, H, d, "state");
  decay_state(state_out, B, H, d, "state_out");
  if (out) row(*out, B, H, d, "out");
  same_device(q, {&k, &v, &log_decay, &state, opt(out), opt(state_out)});
  Here here(q);
  Tensor o = out ? *out : make({B, H, d}, at::kBFloat16, q);
  Tensor so = state_out ? *state_out : state;
  const int64_t s[8] = {q.stride(0), q.stride(1), k.stride(0), k.stride(1), v.stride(0), v.stride(1), o.stride(0),
                        o.stride(1)};
  check(sagesla_linear_decay_step(ptr(q), ptr(k), ptr(v), (const float*)ptr(log_decay), (const float*)ptr(state),
                                  (float)scale, ptr(o), (float*)ptr(so), small(B, "B"), small(H, "H"), small(Hk, "H"),
                                  small(d, "d"), s, here.st),
        "sagesla_linear_decay_step");
  return py::make_tuple(o, so);
}

}  // namespace

PYBIND11_MODULE(_layer, m) {
  m.def("w8a8_token_quant", &w8a8_token_quant);
  m.def("w8a8_token_gemm", &w8a8_token_gemm);
  m.def("w8a8_token_linear", &w8a8_token_linear);
  m.def("qk_norm_rope", &qk_norm_rope);
  m.def("qk_norm_rope_bwd", &qk_norm_rope_bwd);
  m.def("linear_decay", &linear_decay);
  m.def("linear_decay_step", &linear_decay_step);
}
