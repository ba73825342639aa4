// layer_abi.cu -- C entry points of what stands before and beside the experts in
// a layer: the RMS norm, the router's choice and the products with an epilogue;
// argument checks and launches.
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>
#include <mutex>

#include "abi_util.h"
#include "internal.h"

using namespace moe;

namespace {

// Sizes and choices shared by the two routing entry points.
int check_route(int dtype, int T, int E, int K, int scores, int renormalize, float scale) {
  if (T < 0 || E <= 0 || K <= 0 || elem_bytes(dtype) == 0 ||
      (scores != MOE_SCORE_SOFTMAX && scores != MOE_SCORE_SIGMOID) ||
      (renormalize != 0 && renormalize != 1) || !std::isfinite(scale))
    return MOE_ERR_INVALID_ARG;
  if (E > 1024 || K > 32) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Elements of a row that TMA's 32-bit coordinates count in bytes, and rows of a
// tile index.
constexpr int kMaxElements = (1 << 30) - 4096;
constexpr int kMaxRows = 0x7fffffff - 512;
// Elements of a sum: a tile's epilogue waits for all of its K steps, 0.3 us each,
// with a limit of two seconds.
constexpr int kMaxSum = 1 << 27;

// What the products' forms hold at once on the current device, looked up once
// per device.
LinearHeld linear_held_here() {
  static std::mutex mu;
  static bool known[64];
  static LinearHeld held[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    cudaGetLastError();
    return LinearHeld{};
  }
  std::lock_guard<std::mutex> lk(mu);
  if (!known[dev]) {
    held[dev] = linear_held();
    known[dev] = true;
  }
  return held[dev];
}

int check_linear(int M, int N, int K, int act, int out_dtype) {
  if (M < 0 || N <= 0 || K <= 0 || act < MOE_LINEAR_NONE || act > MOE_LINEAR_SWIGLU ||
      elem_bytes(out_dtype) == 0)
    return MOE_ERR_INVALID_ARG;
  if (M > kMaxRows || N > kMaxElements / 2 || K > kMaxSum) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

LinearArgs linear_args(int M, int N, int K, int act, void* out, int out_dtype, int32_t* status) {
  LinearArgs a;
  std::memset(&a, 0, sizeof(a));
  a.M = M;
  a.N = act == MOE_LINEAR_SWIGLU ? 2 * N : N;
  a.K = K;
  a.epi.out = out;
  a.epi.cols = N;
  a.epi.act = act;
  a.epi.out_bf16 = out_dtype == MOE_BF16;
  a.status = status;
  return a;
}

// The product of a.M rows, a.N weight rows and a.K elements, its operands as
// `layout` says; `force`: null, or the form to use instead of the choice by the
// sizes.
int run_linear(LinearArgs a, const void* x, const void* w, LinearLayout layout, cudaStream_t s,
               const LinearForm* force = nullptr) {
  const int es = a.epi.out_bf16 ? 2 : 4;
  if (!x || !w || !a.epi.out || !aligned(x, 16) || !aligned(w, 16) || !aligned(a.epi.out, es) ||
      !aligned(a.epi.residual, es) || !aligned(a.epi.preact, 2) || !words(a.epi.bias, a.status))
    return MOE_ERR_INVALID_ARG;
  // rows of an operand start on 16 bytes
  const int x_row = layout == kColsCols ? a.M : a.K, w_row = layout == kRowsRows ? a.K : a.N;
  if (x_row % 8 != 0 || w_row % 8 != 0) return MOE_ERR_UNSUPPORTED;
  if ((static_cast<long long>(a.M) / 128 + 1) * (a.N / 32 + 1) > 0x3fffffffll)
    return MOE_ERR_UNSUPPORTED;  // tile indexes are 32-bit
  a.epi.wide = a.epi.cols % 8 == 0 && aligned(a.epi.out, 16) && aligned(a.epi.residual, 16) &&
               aligned(a.epi.preact, 16) && aligned(a.epi.bias, 16);
  if (a.timeout_ns == 0) a.timeout_ns = kWaitTimeoutNs;
  const int sms = device_sm_count();
  // Few rows: the kernel for them.
  const bool few = layout == kRowsRows && a.M <= kRowsMax;
  if (force != nullptr ? force->bn == 16 : few)
    return cuda_status(launch_linear_rows(a, x, w, sms, s));
  const LinearForm f = force != nullptr ? *force : linear_form(a, sms, linear_held_here());
  const bool gated = a.epi.act == MOE_LINEAR_SWIGLU;
  a.short_a = !f.pair && layout != kColsCols && a.M <= 32;
  CUtensorMap tm_a, tm_b;
  int rc = layout == kColsCols ? make_byte_map(&tm_a, x, 2ll * a.M, a.K, 128, 64)
                               : make_byte_map(&tm_a, x, 2ll * a.K, a.M, 128, a.short_a ? 32 : 128);
  if (rc == MOE_OK)
    rc = layout == kRowsRows
             ? make_byte_map(&tm_b, w, 2ll * a.K, a.N, 128, f.pair || gated ? f.bn / 2 : f.bn)
             : make_byte_map(&tm_b, w, 2ll * a.N, a.K, 128, 64);
  if (rc != MOE_OK) return rc;
  return cuda_status(launch_linear(a, layout, f, tm_a, tm_b, s));
}

}  // namespace

extern "C" {

int moe_rms_norm(const void* x, const void* residual, const void* weight, int dtype,
                 int weight_dtype, int T, int H, float eps, void* sum, void* out, uint8_t* codes,
                 float* scale, float* rstd, void* stream) {
  const int es = elem_bytes(dtype), ws = elem_bytes(weight_dtype);
  if (T < 0 || H <= 0 || es == 0 || ws == 0 || !(eps >= 0.0f) || !std::isfinite(eps))
    return MOE_ERR_INVALID_ARG;
  if (H > kMaxColumns) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!x || !weight || (!out && !codes) || !codes != !scale || !aligned(x, es) ||
      !aligned(residual, es) || !aligned(weight, ws) || !aligned(sum, es) || !aligned(out, es) ||
      !words(scale, rstd))
    return MOE_ERR_INVALID_ARG;
  RmsNormArgs a;
  a.T = T;
  a.H = H;
  a.x = x;
  a.residual = residual;
  a.weight = weight;
  a.w_bf16 = weight_dtype == MOE_BF16;
  a.eps = eps;
  a.sum_out = sum;
  a.out = out;
  a.codes = codes;
  a.scale = scale;
  a.rstd = rstd;
  return cuda_status(launch_rms_norm(a, dtype, as_stream(stream)));
}

size_t moe_rms_norm_backward_scratch_bytes(int T, int H) {
  if (T <= 0 || H <= 0 || H > kMaxColumns) return 0;
  return static_cast<size_t>(rms_norm_grad_parts(T, H, device_sm_count())) * H * sizeof(float);
}

int moe_rms_norm_backward(const void* grad_out, const void* h, const void* weight,
                          const float* rstd, const void* grad_sum, int dtype, int weight_dtype,
                          int T, int H, void* grad_x, float* grad_weight, void* scratch,
                          size_t scratch_bytes, void* stream) {
  const int es = elem_bytes(dtype), ws = elem_bytes(weight_dtype);
  if (T < 0 || H <= 0 || es == 0 || ws == 0) return MOE_ERR_INVALID_ARG;
  if (H > kMaxColumns) return MOE_ERR_UNSUPPORTED;
  if (!words(rstd, grad_weight, scratch)) return MOE_ERR_INVALID_ARG;
  if (T == 0) {
    if (grad_weight == nullptr) return MOE_OK;
    return cuda_status(cudaMemsetAsync(grad_weight, 0, static_cast<size_t>(H) * sizeof(float),
                                       as_stream(stream)));
  }
  if (!grad_out || !h || !weight || !rstd || !grad_x || !aligned(grad_out, es) ||
      !aligned(h, es) || !aligned(weight, ws) || !aligned(grad_sum, es) || !aligned(grad_x, es))
    return MOE_ERR_INVALID_ARG;
  const int sms = device_sm_count();
  if (grad_weight != nullptr) {
    const size_t need = static_cast<size_t>(rms_norm_grad_parts(T, H, sms)) * H * sizeof(float);
    if (scratch == nullptr || scratch_bytes < need) return MOE_ERR_WORKSPACE;
  }
  RmsNormGradArgs a;
  a.T = T;
  a.H = H;
  a.dy = grad_out;
  a.h = h;
  a.weight = weight;
  a.w_bf16 = weight_dtype == MOE_BF16;
  a.rstd = rstd;
  a.dsum = grad_sum;
  a.dx = grad_x;
  a.part = grad_weight != nullptr ? static_cast<float*>(scratch) : nullptr;
  a.dw = grad_weight;
  return cuda_status(launch_rms_norm_grad(a, dtype, sms, as_stream(stream)));
}

int moe_route_tokens(const void* logits, int logit_dtype, const float* bias, int T, int E, int K,
                     int scores, int num_groups, int topk_groups, int group_scores,
                     int renormalize, float scale, int32_t* topk_ids, float* topk_weights,
                     int32_t* dev_status, void* stream) {
  const int rc = check_route(logit_dtype, T, E, K, scores, renormalize, scale);
  if (rc != MOE_OK) return rc;
  if (num_groups <= 0 || topk_groups <= 0 || topk_groups > num_groups || E % num_groups != 0 ||
      (group_scores != MOE_GROUP_TOP2 && group_scores != MOE_GROUP_MAX) ||
      K > topk_groups * (E / num_groups))
    return MOE_ERR_INVALID_ARG;
  if (num_groups > 32) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!logits || !topk_ids || !topk_weights || !aligned(logits, elem_bytes(logit_dtype)) ||
      !words(bias, topk_ids, topk_weights, dev_status))
    return MOE_ERR_INVALID_ARG;
  RouteTokensArgs a;
  a.logits = logits;
  a.bf16 = logit_dtype == MOE_BF16;
  a.bias = bias;
  a.T = T;
  a.E = E;
  a.K = K;
  a.groups = num_groups;
  a.topk_groups = topk_groups;
  a.softmax = scores == MOE_SCORE_SOFTMAX;
  a.top2 = group_scores == MOE_GROUP_TOP2;
  a.renormalize = renormalize;
  a.scale = scale;
  a.ids = topk_ids;
  a.weights = topk_weights;
  a.status = dev_status;
  return cuda_status(launch_route_tokens(a, as_stream(stream)));
}

int moe_route_tokens_backward(const float* grad_weights, const void* logits, int logit_dtype,
                              const int32_t* topk_ids, int T, int E, int K, int scores,
                              int renormalize, float scale, void* grad_logits,
                              int32_t* dev_status, void* stream) {
  const int rc = check_route(logit_dtype, T, E, K, scores, renormalize, scale);
  if (rc != MOE_OK || T == 0) return rc;
  const int es = elem_bytes(logit_dtype);
  if (!grad_weights || !logits || !topk_ids || !grad_logits || !aligned(logits, es) ||
      !aligned(grad_logits, es) || !words(grad_weights, topk_ids, dev_status))
    return MOE_ERR_INVALID_ARG;
  RouteTokensGradArgs a;
  a.grad = grad_weights;
  a.logits = logits;
  a.bf16 = logit_dtype == MOE_BF16;
  a.ids = topk_ids;
  a.T = T;
  a.E = E;
  a.K = K;
  a.softmax = scores == MOE_SCORE_SOFTMAX;
  a.renormalize = renormalize;
  a.scale = scale;
  a.dlogits = grad_logits;
  a.status = dev_status;
  return cuda_status(launch_route_tokens_grad(a, as_stream(stream)));
}

int moe_linear(const void* x, const void* w, const float* bias, const void* residual, int M, int N,
               int K, int activation, void* out, int out_dtype, void* preact, int32_t* dev_status,
               void* stream) {
  const int rc = check_linear(M, N, K, activation, out_dtype);
  if (rc != MOE_OK || M == 0) return rc;
  LinearArgs a = linear_args(M, N, K, activation, out, out_dtype, dev_status);
  a.epi.bias = bias;
  a.epi.residual = residual;
  a.epi.preact = static_cast<__nv_bfloat16*>(preact);
  return run_linear(a, x, w, kRowsRows, as_stream(stream));
}

size_t moe_linear_backward_act_scratch_bytes(int M, int N, int activation) {
  if (check_linear(M, N, 1, activation, MOE_BF16) != MOE_OK || M == 0) return 0;
  const int rows = activation == MOE_LINEAR_SWIGLU ? 2 * N : N;
  return static_cast<size_t>(linear_grad_parts(M, rows, activation, device_sm_count())) * rows *
         sizeof(float);
}

int moe_linear_backward_act(const void* grad_out, const void* preact, int M, int N, int activation,
                            void* grad_preact, float* grad_bias, void* scratch,
                            size_t scratch_bytes, void* stream) {
  const int rc = check_linear(M, N, 1, activation, MOE_BF16);
  if (rc != MOE_OK) return rc;
  if (!words(grad_bias, scratch)) return MOE_ERR_INVALID_ARG;
  const int rows = activation == MOE_LINEAR_SWIGLU ? 2 * N : N;
  if (M == 0) {
    if (grad_bias == nullptr) return MOE_OK;
    return cuda_status(cudaMemsetAsync(grad_bias, 0, static_cast<size_t>(rows) * sizeof(float),
                                       as_stream(stream)));
  }
  // with no activation grad_preact is grad_out, and there is only the bias
  const bool none = activation == MOE_LINEAR_NONE;
  if (!grad_out || (!none && (!preact || !grad_preact)) || (none && !grad_bias) ||
      !aligned(grad_out, 2) || !aligned(preact, 2) || !aligned(grad_preact, 2))
    return MOE_ERR_INVALID_ARG;
  const int sms = device_sm_count();
  if (grad_bias != nullptr) {
    const size_t need =
        static_cast<size_t>(linear_grad_parts(M, rows, activation, sms)) * rows * sizeof(float);
    if (scratch == nullptr || scratch_bytes < need) return MOE_ERR_WORKSPACE;
  }
  LinearGradArgs a;
  a.M = M;
  a.N = rows;
  a.act = activation;
  a.dy = static_cast<const __nv_bfloat16*>(grad_out);
  a.preact = static_cast<const __nv_bfloat16*>(preact);
  a.dz = none ? nullptr : static_cast<__nv_bfloat16*>(grad_preact);
  a.part = grad_bias != nullptr ? static_cast<float*>(scratch) : nullptr;
  a.db = grad_bias;
  return cuda_status(launch_linear_grad(a, sms, as_stream(stream)));
}

int moe_linear_backward_input(const void* grad_preact, const void* w, int M, int N, int K,
                              void* grad_x, int out_dtype, int32_t* dev_status, void* stream) {
  const int rc = check_linear(M, K, N, MOE_LINEAR_NONE, out_dtype);
  if (rc != MOE_OK || M == 0) return rc;
  return run_linear(linear_args(M, K, N, MOE_LINEAR_NONE, grad_x, out_dtype, dev_status),
                    grad_preact, w, kRowsCols, as_stream(stream));
}

int moe_linear_backward_weight(const void* grad_preact, const void* x, int M, int N, int K,
                               void* grad_w, int out_dtype, int accumulate, int32_t* dev_status,
                               void* stream) {
  if (accumulate != 0 && accumulate != 1) return MOE_ERR_INVALID_ARG;
  if (M < 0 || N <= 0) return MOE_ERR_INVALID_ARG;
  // no rows: the sum is empty
  const int rc = check_linear(N, K, M == 0 ? 1 : M, MOE_LINEAR_NONE, out_dtype);
  if (rc != MOE_OK) return rc;
  if (N > kMaxElements) return MOE_ERR_UNSUPPORTED;  // along the rows of grad_preact
  if (M == 0) {
    if (accumulate) return MOE_OK;
    if (!grad_w || !aligned(grad_w, elem_bytes(out_dtype))) return MOE_ERR_INVALID_ARG;
    return cuda_status(cudaMemsetAsync(grad_w, 0,
                                       static_cast<size_t>(N) * K * elem_bytes(out_dtype),
                                       as_stream(stream)));
  }
  LinearArgs a = linear_args(N, K, M, MOE_LINEAR_NONE, grad_w, out_dtype, dev_status);
  if (accumulate) a.epi.residual = grad_w;
  return run_linear(a, grad_preact, x, kColsCols, as_stream(stream));
}

int moe_test_linear(const void* x, const void* w, int M, int N, int K, int layout, int activation,
                    void* out, int out_dtype, int form, unsigned long long wait_limit_ns,
                    int32_t* dev_status, void* stream) {
  const int rc = check_linear(M, N, K, activation, out_dtype);
  if (rc != MOE_OK) return rc;
  const bool narrow = form == 224;
  if (M == 0 || layout < kRowsRows || layout > kColsCols || form < 0 || (form > 7 && !narrow) ||
      (layout != kRowsRows && activation == MOE_LINEAR_SWIGLU) ||
      (wait_limit_ns != 0 && (wait_limit_ns < 1000000ull || wait_limit_ns > 2000000000ull)))
    return MOE_ERR_INVALID_ARG;
  // {weight rows of a tile, pair, splits} of the forms
  static const int kForms[8][3] = {{64, 0, 1}, {128, 0, 1}, {64, 0, 2},  {64, 0, 4},
                                   {64, 0, 8}, {16, 0, 1},  {256, 1, 1}, {128, 1, 1}};
  LinearForm f;
  f.bn = narrow ? 224 : kForms[form][0];
  f.pair = narrow || kForms[form][1] != 0;
  f.splits = narrow ? 1 : kForms[form][2];
  if (layout == kColsCols && M > kMaxElements) return MOE_ERR_UNSUPPORTED;
  // few rows: no waits and one layout; a split has K steps of 64 for all its CTAs;
  // 224 columns: one accumulator
  if ((f.bn == 16 && (M > kRowsMax || wait_limit_ns != 0 || layout != kRowsRows)) ||
      (narrow && (out_dtype != MOE_BF16 || K > kMostOfAccumulator)) ||
      (K + 63) / 64 < f.splits)
    return MOE_ERR_UNSUPPORTED;
  LinearArgs a = linear_args(M, N, K, activation, out, out_dtype, dev_status);
  a.timeout_ns = wait_limit_ns;
  a.starve = wait_limit_ns != 0;
  const int bm = f.pair ? 256 : 128;
  const int bn = activation == MOE_LINEAR_SWIGLU ? f.bn / 2 : f.bn;
  const long long tiles =
      (static_cast<long long>(M) + bm - 1) / bm * ((static_cast<long long>(N) + bn - 1) / bn);
  if (tiles * f.splits > 0x1fffffffll) return MOE_ERR_UNSUPPORTED;
  const int slots = f.pair ? linear_held_here().pairs : device_sm_count();
  if (slots <= 0) return MOE_ERR_CUDA;
  const long long in_flight = f.splits > 1 ? tiles : tiles < slots ? tiles : slots;
  f.grid = static_cast<int>(in_flight * f.splits * (f.pair ? 2 : 1));
  return run_linear(a, x, w, static_cast<LinearLayout>(layout), as_stream(stream), &f);
}

}  // extern "C"
