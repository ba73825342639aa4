// ops_abi.cu -- C entry points of the token permutation, the 128-column fp8
// quantiser and the block-scaled products: argument checks and launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstring>
#include <mutex>

#include "internal.h"

using namespace moe;

namespace {

int cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }

// Element bytes of `dtype`, 0 when it is not one of the two row types (or,
// with `codes`, of the three).
int elem_bytes(int dtype, bool codes = false) {
  if (dtype == MOE_F32) return 4;
  if (dtype == MOE_BF16) return 2;
  return codes && dtype == MOE_E4M3 ? 1 : 0;
}

bool aligned(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

// int32 and fp32 arguments, which the kernels access as 4-byte words.
template <typename... P>
bool words(const P*... p) {
  return (aligned(p, 4) && ...);
}

// Columns of a row: the kernels count them in 32 bits and step past the last
// one by up to one CTA's worth (2048).
constexpr int kMaxColumns = 0x7fffffff - 4096;

// Sizes shared by the four permutation entry points; cap is an int32 slot
// count in the lists.
int check_list(int T, int H, int K, size_t cap, int es) {
  if (T < 0 || H <= 0 || K <= 0 || es == 0) return MOE_ERR_INVALID_ARG;
  if (static_cast<long long>(T) * K >= (1ll << 30) || cap > 0x7fffffffull || H > kMaxColumns)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

int check_gemm(int E, int N, int K, int out_dtype) {
  if (E <= 0 || N <= 0 || K <= 0 || elem_bytes(out_dtype) == 0) return MOE_ERR_INVALID_ARG;
  // TMA rows start on 16 bytes, and row coordinates are 32-bit
  if (K % 16 != 0 || K > kMaxColumns || static_cast<long long>(E) * N >= (1ll << 31) - 256)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// What the product's forms hold at once on the current device, looked up once
// per device.
Fp8bHeld held_clusters() {
  static std::mutex mu;
  static bool known[64];
  static Fp8bHeld held[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    cudaGetLastError();
    return Fp8bHeld{};
  }
  std::lock_guard<std::mutex> lk(mu);
  if (!known[dev]) {
    held[dev] = fp8b_held();
    known[dev] = true;
  }
  return held[dev];
}

// `force`: null, or the form to use instead of the choice by the sizes.
int run_gemm(Fp8bArgs a, const uint8_t* x, long long rows, const uint8_t* w, int out_dtype,
             cudaStream_t s, const Fp8bForm* force = nullptr) {
  const int es = elem_bytes(out_dtype);
  if (!x || !a.a_scale || !w || !a.w_scale || !a.out || !aligned(x, 16) || !aligned(w, 16) ||
      !words(a.a_scale, a.w_scale, a.num_blocks, a.status) || !aligned(a.out, es))
    return MOE_ERR_INVALID_ARG;
  a.k_tiles = (a.K + 127) / 128;
  a.n_scales = (a.N + 127) / 128;
  a.cap = rows;
  a.out_bf16 = out_dtype == MOE_BF16;
  a.wide_out = (static_cast<long long>(a.N) * es) % 16 == 0 && aligned(a.out, 16);
  if (a.timeout_ns == 0) a.timeout_ns = kWaitTimeoutNs;
  // tile indexes are 32-bit
  if (static_cast<long long>(a.max_blocks) * a.subs * ((a.N + 63) / 64) > 0x3fffffffll)
    return MOE_ERR_UNSUPPORTED;
  // Few rows: the kernel for them, as long as latency counts.  From 64 MB of
  // weights on both stream at HBM's rate and the tiles of the other one read a
  // fewer times (us, 8 rows of 16384 x 7168: 28.4 and 23.4; 1 row of 16384 x
  // 4096: 16.7 and 15.4; 8 rows of 4096 x 7168: 10.3 and 11.3).
  const bool few = a.block_info == nullptr && a.M <= kRowsMax &&
                   static_cast<long long>(a.N) * a.K <= (64ll << 20);
  if (force != nullptr ? force->bn == 16 : few)
    return cuda_status(launch_fp8b_rows(a, x, w, device_sm_count(), s));
  const Fp8bForm f = force != nullptr ? *force : fp8b_form(a, device_sm_count(), held_clusters());
  Fp8bMaps maps;
  int rc = make_byte_map(&maps.a, x, a.K, rows, 128, 128);
  if (rc == MOE_OK) rc = make_byte_map(&maps.a_short, x, a.K, rows, 128, 32);
  if (rc == MOE_OK)
    rc = make_byte_map(&maps.b, w, a.K, static_cast<long long>(a.E) * a.N, 128, f.bn);
  if (rc != MOE_OK) return rc;
  return cuda_status(launch_fp8b_gemm(a, f, maps, s));
}

Fp8bArgs plain_args(const float* a_scale, const float* w_scale, int M, int N, int K, void* out,
                    int32_t* status) {
  Fp8bArgs g;
  std::memset(&g, 0, sizeof(g));
  g.M = M;
  g.N = N;
  g.K = K;
  g.E = 1;
  g.max_blocks = M / 128 + (M % 128 != 0);
  g.subs = 1;
  g.block_m = 128;
  g.a_scale = a_scale;
  g.w_scale = w_scale;
  g.out = out;
  g.status = status;
  return g;
}

}  // namespace

extern "C" {

int moe_permute_tokens(const void* x, int dtype, int T, int H, int K, const int32_t* inv_perm,
                       const int32_t* sorted_ids, size_t cap, void* x_sorted,
                       int32_t* dev_status, void* stream) {
  const int es = elem_bytes(dtype, true);
  const int rc = check_list(T, H, K, cap, es);
  if (rc != MOE_OK || T == 0) return rc;
  if (!x || !inv_perm || !sorted_ids || !x_sorted || !aligned(x, es) || !aligned(x_sorted, es) ||
      !words(inv_perm, sorted_ids, dev_status))
    return MOE_ERR_INVALID_ARG;
  return cuda_status(launch_permute(x, T, static_cast<long long>(H) * es, K, inv_perm, sorted_ids,
                                    static_cast<long long>(cap), x_sorted, dev_status,
                                    as_stream(stream)));
}

int moe_permute_tokens_backward(const void* grad_sorted, int dtype, int T, int H, int K,
                                const int32_t* inv_perm, size_t cap, void* grad_x,
                                int32_t* dev_status, void* stream) {
  const int es = elem_bytes(dtype);
  const int rc = check_list(T, H, K, cap, es);
  if (rc != MOE_OK || T == 0) return rc;
  if (!grad_sorted || !inv_perm || !grad_x || !aligned(grad_sorted, es) || !aligned(grad_x, es) ||
      !words(inv_perm, dev_status))
    return MOE_ERR_INVALID_ARG;
  return cuda_status(launch_unpermute(grad_sorted, dtype, nullptr, T, K, H, inv_perm,
                                      static_cast<long long>(cap), grad_x, dev_status,
                                      as_stream(stream)));
}

int moe_unpermute_tokens(const void* y, int dtype, int T, int H, int K, const float* topk_weights,
                         const int32_t* inv_perm, size_t cap, void* out, int32_t* dev_status,
                         void* stream) {
  const int es = elem_bytes(dtype);
  const int rc = check_list(T, H, K, cap, es);
  if (rc != MOE_OK || T == 0) return rc;
  if (!y || !topk_weights || !inv_perm || !out || !aligned(y, es) || !aligned(out, es) ||
      !words(topk_weights, inv_perm, dev_status))
    return MOE_ERR_INVALID_ARG;
  return cuda_status(launch_unpermute(y, dtype, topk_weights, T, K, H, inv_perm,
                                      static_cast<long long>(cap), out, dev_status,
                                      as_stream(stream)));
}

int moe_unpermute_tokens_backward(const void* grad_out, const void* y, int dtype, int T, int H,
                                  int K, const float* topk_weights, const int32_t* inv_perm,
                                  const int32_t* sorted_ids, size_t cap, void* grad_y,
                                  float* grad_weights, int32_t* dev_status, void* stream) {
  const int es = elem_bytes(dtype);
  const int rc = check_list(T, H, K, cap, es);
  if (rc != MOE_OK || T == 0) return rc;
  if (!grad_out || !y || !topk_weights || !inv_perm || !sorted_ids || !grad_y || !grad_weights ||
      !aligned(grad_out, es) || !aligned(y, es) || !aligned(grad_y, es) ||
      !words(topk_weights, inv_perm, sorted_ids, grad_weights, dev_status))
    return MOE_ERR_INVALID_ARG;
  return cuda_status(launch_unpermute_backward(
      grad_out, y, dtype, topk_weights, T, K, H, inv_perm, sorted_ids,
      static_cast<long long>(cap), grad_y, grad_weights, dev_status, as_stream(stream)));
}

int moe_quantize_fp8_block(const void* x, int x_dtype, int T, int H, int gated, uint8_t* xq,
                           float* scale, void* stream) {
  const int es = elem_bytes(x_dtype);
  if (T < 0 || H <= 0 || es == 0 || (gated != 0 && gated != 1)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  // blocks are counted in 32 bits, and so are their CTAs
  if (static_cast<long long>(T) * ((H + 127ll) / 128) >= (1ll << 31) || H > kMaxColumns)
    return MOE_ERR_UNSUPPORTED;
  if (!x || !xq || !scale || !aligned(x, es) || !words(scale)) return MOE_ERR_INVALID_ARG;
  return cuda_status(
      launch_quantize_block(x, x_dtype, T, H, gated, xq, scale, as_stream(stream)));
}

int moe_gemm_fp8_block(const uint8_t* a, const float* a_scale, const uint8_t* w,
                       const float* w_scale, int M, int N, int K, void* out, int out_dtype,
                       int32_t* dev_status, void* stream) {
  const int rc = check_gemm(1, N, K, out_dtype);
  if (rc != MOE_OK || M < 0) return rc != MOE_OK ? rc : MOE_ERR_INVALID_ARG;
  if (M == 0) return MOE_OK;
  return run_gemm(plain_args(a_scale, w_scale, M, N, K, out, dev_status), a, M, w, out_dtype,
                  as_stream(stream));
}

int moe_grouped_gemm_fp8_block(const uint8_t* a, const float* a_scale, const uint8_t* w,
                               const float* w_scale, int E, int N, int K, size_t cap, int block_m,
                               const int32_t* block_info, const int32_t* num_blocks, void* out,
                               int out_dtype, int32_t* dev_status, void* stream) {
  const int rc = check_gemm(E, N, K, out_dtype);
  if (rc != MOE_OK) return rc;
  if (block_m != 16 && block_m != 32 && block_m != 64 && block_m != 128 && block_m != 256)
    return MOE_ERR_INVALID_ARG;
  if (cap > 0x7fffffffull - 256) return MOE_ERR_UNSUPPORTED;
  if (cap / block_m == 0) return MOE_OK;
  if (!block_info || !num_blocks || !aligned(block_info, 16)) return MOE_ERR_INVALID_ARG;
  Fp8bArgs g;
  std::memset(&g, 0, sizeof(g));
  g.N = N;
  g.K = K;
  g.E = E;
  g.block_info = block_info;
  g.num_blocks = num_blocks;
  g.max_blocks = static_cast<int>(cap / block_m);
  g.subs = block_m > 128 ? block_m / 128 : 1;
  g.block_m = block_m;
  g.a_scale = a_scale;
  g.w_scale = w_scale;
  g.out = out;
  g.status = dev_status;
  return run_gemm(g, a, static_cast<long long>(cap), w, out_dtype, as_stream(stream));
}

int moe_test_gemm_fp8_block(const uint8_t* a, const float* a_scale, const uint8_t* w,
                            const float* w_scale, int M, int N, int K, void* out, int out_dtype,
                            int form, unsigned long long wait_limit_ns, int32_t* dev_status,
                            void* stream) {
  const int rc = check_gemm(1, N, K, out_dtype);
  if (rc != MOE_OK) return rc;
  // the form's 16 is what a failure-path run holds back
  const bool scales_only = form >= 16 && wait_limit_ns != 0;
  if (scales_only) form -= 16;
  if (M <= 0 || form < 0 || form > 5) return MOE_ERR_INVALID_ARG;
  // the form without pipelines has no waits, and takes few rows
  if (form == 5 && (M > kRowsMax || wait_limit_ns != 0)) return MOE_ERR_UNSUPPORTED;
  if (wait_limit_ns != 0 && (wait_limit_ns < 1000000ull || wait_limit_ns > 2000000000ull))
    return MOE_ERR_INVALID_ARG;
  Fp8bArgs g = plain_args(a_scale, w_scale, M, N, K, out, dev_status);
  g.timeout_ns = wait_limit_ns;
  g.starve = wait_limit_ns == 0 ? kStarveNone : scales_only ? kStarveScales : kStarveAll;
  // {weight rows of a tile, mode, splits} of forms 0 to 4
  static const int kForms[6][3] = {{64, 0, 1}, {128, 0, 1}, {64, 1, 2},
                                   {64, 1, 4}, {64, 1, 8},  {16, 0, 1}};
  Fp8bForm f;
  f.bn = kForms[form][0];
  f.mode = kForms[form][1];
  f.splits = kForms[form][2];
  const long long tiles = static_cast<long long>(g.max_blocks) * ((N + f.bn - 1) / f.bn);
  if (tiles * f.splits > 0x3fffffffll) return MOE_ERR_UNSUPPORTED;
  const int sms = device_sm_count();
  f.grid = static_cast<int>(f.splits > 1 ? tiles * f.splits : tiles < sms ? tiles : sms);
  return run_gemm(g, a, M, w, out_dtype, as_stream(stream), &f);
}

}  // extern "C"
