// linear_grad.cu -- the step between a product's output gradient and the products
// of its own gradients: dz = dy * act'(z) with z as the forward pass kept it, and
// the bias gradient, the sums of dz's columns.
//
//   silu   dz = dy s (1 + z (1 - s)),  s = 1 / (1 + e^-z)
//   gelu   dz = dy (Phi(z) + z phi(z)),  Phi and phi of the normal distribution
//   swiglu dgate = dy u s (1 + g (1 - s)), dup = dy g s
//
// dz is rounded to bf16, the type of the operands of the products that follow;
// the column sums are of the unrounded values: a thread adds eight columns of
// every 8 x parts-th row, a CTA its eight row lanes, add_parts the CTAs, all in a fixed
// order.  One read of dy and z and one write of dz bound SiLU; GELU's arithmetic adds to them
// (its kernel fills 56 % of the issue slots while its warps wait for HBM and for the arithmetic
// pipes by turns), and the sums of the columns take a kernel of their own, 2.5 us.  GB300,
// operands from HBM, us (at the copy rate of 6.8 TB/s): 4096 x 4096 SiLU 18.4 (14.8), with the
// bias's gradient 20.7, GELU 21.5 and 23.8, SwiGLU of 2 x 2048 columns 16.5 and 19.3 (12.3),
// 8192 x 7168 SiLU 56 (51.8).
#include <cuda_bf16.h>

#include <algorithm>

#include "internal.h"
#include "linear_epi.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kVec = 8;
constexpr int kLanes = 32;     // column groups of a CTA: 256 columns
constexpr int kRowLanes = 8;
constexpr int kThreads = kLanes * kRowLanes;
// CTAs per SM, what the registers leave: with two rows on a thread's way, one for SwiGLU's
// three operands (4096 x 4096 SiLU, us with the bias's gradient: one row 22.8, two 21.0, twice
// the CTAs 21.4; SwiGLU, 4096 x 2 x 2048: one row 19.1, two 21.2, twice the CTAs 19.7).
constexpr int per_sm(bool gated) { return gated ? 3 : 4; }

// Columns [c, c + 8) of a row of n, zero past its end.
template <bool WIDE>
__device__ __forceinline__ uint4 load8(const __nv_bfloat16* row, int c, int n) {
  if constexpr (WIDE) return *reinterpret_cast<const uint4*>(row + c);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t lo = 0, hi = 0;
    if (c + 2 * i < n) lo = __bfloat16_as_ushort(row[c + 2 * i]);
    if (c + 2 * i + 1 < n) hi = __bfloat16_as_ushort(row[c + 2 * i + 1]);
    w[i] = lo | hi << 16;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
constexpr int kPairs = kVec / 2;
__device__ __forceinline__ void values(uint4 q, float2 (&v)[kPairs]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < kPairs; ++i)
    v[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}

template <bool WIDE>
__device__ __forceinline__ void store8(__nv_bfloat16* row, int c, int n,
                                       const float2 (&v)[kPairs]) {
  if constexpr (WIDE) {
    *reinterpret_cast<uint4*>(row + c) =
        make_uint4(bf16_pair(v[0].x, v[0].y), bf16_pair(v[1].x, v[1].y),
                   bf16_pair(v[2].x, v[2].y), bf16_pair(v[3].x, v[3].y));
  } else {
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      if (c + 2 * i < n) row[c + 2 * i] = __float2bfloat16_rn(v[i].x);
      if (c + 2 * i + 1 < n) row[c + 2 * i + 1] = __float2bfloat16_rn(v[i].y);
    }
  }
}

// z within fp32's finite values
__device__ __forceinline__ float2 finite(float2 z) {
  return make_float2(fmaxf(fminf(z.x, kLargest), -kLargest),
                     fmaxf(fminf(z.y, kLargest), -kLargest));
}
// SiLU'(z) given s = sigmoid(z); z finite
__device__ __forceinline__ float2 silu_slope(float2 z, float2 s) {
  const float2 rest = __ffma2_rn(s, both(-1.0f), both(1.0f));
  return __fmul2_rn(s, __ffma2_rn(z, rest, both(1.0f)));
}
// Phi(z) + z phi(z), 1 and 0 at the infinities
__device__ __forceinline__ float2 gelu_slope(float2 z) {
  float2 e;
  const float2 h = normal_tail(z, e);
  const float2 near = make_float2(fmaxf(fminf(z.x, kTailEnd), -kTailEnd),
                                  fmaxf(fminf(z.y, kTailEnd), -kTailEnd));
  const float2 all = make_float2(z.x >= 0.0f ? 1.0f - h.x : h.x, z.y >= 0.0f ? 1.0f - h.y : h.y);
  return __ffma2_rn(__fmul2_rn(near, both(0.39894228f)), e, all);
}

template <bool WIDE, bool GATED>
__global__ void __launch_bounds__(kThreads, per_sm(GATED))
    linear_grad_kernel(const __grid_constant__ LinearGradArgs a) {
  constexpr int kAtOnce = WIDE && !GATED ? 2 : 1;  // rows of a thread whose words are on their way
  __shared__ __align__(8) float s_sum[kRowLanes][kLanes * kVec];
  pdl_wait();
  pdl_launch_dependents();
  const int cols = GATED ? a.N / 2 : a.N;  // of dy
  const int x = threadIdx.x % kLanes, y = threadIdx.x / kLanes;
  const long long c0 = (static_cast<long long>(blockIdx.x) * kLanes + x) * kVec;
  const int c = static_cast<int>(c0 < cols ? c0 : cols);
  float2 sum[kPairs], sum_up[kPairs];
#pragma unroll
  for (int i = 0; i < kPairs; ++i) sum[i] = sum_up[i] = both(0.0f);
  if (c < cols) {
    const long long step = static_cast<long long>(gridDim.y) * kRowLanes;
    const long long first = static_cast<long long>(blockIdx.y) * kRowLanes + y;
    for (long long m0 = first; m0 < a.M; m0 += kAtOnce * step) {
      uint4 qd[kAtOnce], qz[kAtOnce], qu[GATED ? kAtOnce : 1];
#pragma unroll
      for (int r = 0; r < kAtOnce; ++r) {
        const long long m = m0 + r * step;
        if (m >= a.M) break;
        qd[r] = load8<WIDE>(a.dy + m * cols, c, cols);
        if (a.act != MOE_LINEAR_NONE) qz[r] = load8<WIDE>(a.preact + m * a.N, c, cols);
        if constexpr (GATED) qu[r] = load8<WIDE>(a.preact + m * a.N + cols, c, cols);
      }
#pragma unroll
      for (int r = 0; r < kAtOnce; ++r) {
        const long long m = m0 + r * step;
        if (m >= a.M) break;
        float2 d[kPairs], z[kPairs];
        values(qd[r], d);
        if (a.act != MOE_LINEAR_NONE) values(qz[r], z);
        if constexpr (GATED) {
          float2 u[kPairs];
          values(qu[r], u);
#pragma unroll
          for (int i = 0; i < kPairs; ++i) {
            const float2 s = sigmoid(z[i]);
            const float2 up = __fmul2_rn(d[i], silu(z[i], s));
            d[i] = __fmul2_rn(__fmul2_rn(d[i], u[i]), silu_slope(finite(z[i]), s));
            u[i] = up;
            sum_up[i] = __fadd2_rn(sum_up[i], up);
          }
          if (a.dz != nullptr) store8<WIDE>(a.dz + m * a.N + cols, c, cols, u);
        } else if (a.act == MOE_LINEAR_SILU) {
#pragma unroll
          for (int i = 0; i < kPairs; ++i)
            d[i] = __fmul2_rn(d[i], silu_slope(finite(z[i]), sigmoid(z[i])));
        } else if (a.act == MOE_LINEAR_GELU) {
#pragma unroll
          for (int i = 0; i < kPairs; ++i) d[i] = __fmul2_rn(d[i], gelu_slope(z[i]));
        }
#pragma unroll
        for (int i = 0; i < kPairs; ++i) sum[i] = __fadd2_rn(sum[i], d[i]);
        if (a.dz != nullptr) store8<WIDE>(a.dz + m * a.N, c, cols, d);
      }
    }
  }
  if (a.part == nullptr) return;
  float* part = a.part + static_cast<long long>(blockIdx.y) * a.N;
  for (int h = 0; h < (GATED ? 2 : 1); ++h) {
    if (h > 0) __syncthreads();
#pragma unroll
    for (int i = 0; i < kPairs; ++i)
      *reinterpret_cast<float2*>(&s_sum[y][x * kVec + 2 * i]) = h > 0 ? sum_up[i] : sum[i];
    __syncthreads();
    const long long col = static_cast<long long>(blockIdx.x) * kLanes * kVec + threadIdx.x;
    if (col < cols) {
      float v = 0.0f;
#pragma unroll
      for (int r = 0; r < kRowLanes; ++r) v += s_sum[r][threadIdx.x];
      part[h * static_cast<long long>(cols) + col] = v;
    }
  }
}

static_assert(kThreads == kLanes * kVec, "a thread adds up one column");

int strips(int N, int act) {
  const int cols = act == MOE_LINEAR_SWIGLU ? N / 2 : N;
  return (cols - 1) / (kLanes * kVec) + 1;
}

bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace

// CTAs along the rows: as many as are resident at once.
int linear_grad_parts(int M, int N, int act, int sms) {
  const int most = std::min(65535, (M - 1) / kRowLanes + 1);
  return std::max(1, std::min(most, per_sm(act == MOE_LINEAR_SWIGLU) * sms / strips(N, act)));
}

cudaError_t launch_linear_grad(const LinearGradArgs& a, int sms, cudaStream_t s) {
  const int cols = a.act == MOE_LINEAR_SWIGLU ? a.N / 2 : a.N;
  const int parts = linear_grad_parts(a.M, a.N, a.act, sms);
  const bool wide = cols % kVec == 0 && on16(a.dy) && on16(a.preact) && on16(a.dz);
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg =
      pdl_config(dim3(strips(a.N, a.act), parts), dim3(kThreads), 0, s, attr);
  const bool gated = a.act == MOE_LINEAR_SWIGLU;
  auto* kern = wide ? (gated ? linear_grad_kernel<true, true> : linear_grad_kernel<true, false>)
                    : (gated ? linear_grad_kernel<false, true> : linear_grad_kernel<false, false>);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a);
  if (e != cudaSuccess || a.part == nullptr) return e;
  return launch_add_parts(a.part, parts, a.N, a.db, s);
}

}  // namespace moe
