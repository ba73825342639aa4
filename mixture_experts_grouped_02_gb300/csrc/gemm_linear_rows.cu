// gemm_linear_rows.cu -- the product of gemm_linear.cu for at most eight rows of x
// (decode): streaming the weights once is all there is to do, and what counts is
// how early the loads leave and how few steps follow them.
//
// A CTA owns 16 weight rows (SwiGLU: 8 gate rows and the up rows of the same
// columns) and all of K; its warps take segments of 64 elements in turn and add
// their partial sums through shared memory, in warp order.  The products are
// mma.sync m16n8k16 with the weights as the 16-row operand and the rows of x as
// the 8-column one: no shared memory or TMEM stands between a load and its MMA.
// The K positions inside a segment are dealt to the fragments so that a lane's
// four MMAs take 32 consecutive bytes of a row (both operands the same way, so the
// sum is the same).  mma.sync runs far below the tcgen05 rate, which does not
// matter here.  Row m of x fills column m of the MMA, so a NaN stays in its row.
//
// Bound by HBM.  GB300, weights from HBM, us (at the copy rate of 6.8 TB/s): 1 x 4096 x
// 7168 12.5 (8.6), 8 x 4096 x 7168 13.3 (8.7), 8 x 16384 x 7168 39 (34.6): a launch, one
// trip to HBM and the reduction are 3 to 4 us beside the streaming.  (The weights through
// rings of shared memory: 12.8 and 58.)
#include <cuda_bf16.h>

#include <algorithm>

#include "internal.h"
#include "linear_epi.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kRows = 16;     // weight rows of a CTA
constexpr int kTokens = 8;    // rows of x
constexpr int kMaxWarps = 16;
constexpr int kInFlight = 4;  // segments a warp loads at once
constexpr int kSegment = 64;

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The 16 elements at element k of a row of K (a multiple of 8), zero past K.
__device__ __forceinline__ void load16(const __nv_bfloat16* row, int k, int K, uint4 (&v)[2]) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
    v[h] = k + 8 * h < K ? __ldg(reinterpret_cast<const uint4*>(row + k + 8 * h))
                         : make_uint4(0u, 0u, 0u, 0u);
}

__global__ void __launch_bounds__(kMaxWarps * 32)
    linear_rows_kernel(const __grid_constant__ LinearArgs p, const __nv_bfloat16* __restrict__ x,
                       const __nv_bfloat16* __restrict__ w) {
  constexpr int U = kInFlight;
  __shared__ float s_part[kMaxWarps][kTokens][kRows];
  pdl_wait();
  pdl_launch_dependents();
  // One answer for the CTA, as the word may change while its warps start; it is needed when the
  // sums are done and comes beside the weights.
  __shared__ int s_stop;
  int stop = 0;
  if (threadIdx.x == 0 && p.status != nullptr)
    stop = *reinterpret_cast<volatile int32_t*>(p.status);
  const bool gated = p.epi.act == MOE_LINEAR_SWIGLU;
  const int n0 = blockIdx.x * (gated ? kRows / 2 : kRows);  // the CTA's first output column
  const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  // rows past the last one read that one and are not stored
  const int last = p.epi.cols - 1;
  const long long r0 = min(n0 + g, last);
  const long long r1 = gated ? r0 + p.epi.cols : min(n0 + g + 8, last);
  const __nv_bfloat16* w0 = w + r0 * p.K;
  const __nv_bfloat16* w1 = w + r1 * p.K;
  const __nv_bfloat16* row = x + static_cast<long long>(min(g, p.M - 1)) * p.K;
  const int segments = (p.K - 1) / kSegment + 1;
  float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};

  for (int s0 = warp; s0 < segments; s0 += U * warps) {
    uint4 x0[U][2], x1[U][2], y[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int seg = s0 + u * warps;
      const int k = seg < segments ? seg * kSegment + 16 * t : p.K;
      load16(w0, k, p.K, x0[u]);
      load16(w1, k, p.K, x1[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int seg = s0 + u * warps;
      load16(row, seg < segments && g < p.M ? seg * kSegment + 16 * t : p.K, p.K, y[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (s0 + u * warps >= segments) break;
      const uint32_t a0[8] = {x0[u][0].x, x0[u][0].y, x0[u][0].z, x0[u][0].w,
                              x0[u][1].x, x0[u][1].y, x0[u][1].z, x0[u][1].w};
      const uint32_t a1[8] = {x1[u][0].x, x1[u][0].y, x1[u][0].z, x1[u][0].w,
                              x1[u][1].x, x1[u][1].y, x1[u][1].z, x1[u][1].w};
      const uint32_t b[8] = {y[u][0].x, y[u][0].y, y[u][0].z, y[u][0].w,
                             y[u][1].x, y[u][1].y, y[u][1].z, y[u][1].w};
      // a segment's sum of its own, so that fp32 outputs keep their bits: the
      // tensor core cuts off what it adds to a long sum
      float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int q = 0; q < 4; ++q)
        mma_bf16(d, a0[2 * q], a1[2 * q], a0[2 * q + 1], a1[2 * q + 1], b[2 * q], b[2 * q + 1]);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] += d[i];
    }
  }
  s_part[warp][2 * t][g] = acc[0];
  s_part[warp][2 * t + 1][g] = acc[1];
  s_part[warp][2 * t][g + 8] = acc[2];
  s_part[warp][2 * t + 1][g + 8] = acc[3];
  if (threadIdx.x == 0) s_stop = stop;
  __syncthreads();
  if (s_stop != 0) return;
  __shared__ float s_sum[kTokens][kRows];
  for (int i = threadIdx.x; i < p.M * kRows; i += blockDim.x) {
    float v = 0.0f;
    for (int k = 0; k < warps; ++k) v += s_part[k][i / kRows][i % kRows];
    s_sum[i / kRows][i % kRows] = v;
  }
  __syncthreads();
  const int groups = gated ? 1 : 2;  // of eight output columns
  if (threadIdx.x < p.M * groups) {
    const int m = threadIdx.x / groups, c = 8 * (threadIdx.x % groups);
    float z[1][8], u[1][8];
#pragma unroll
    for (int j = 0; j < 8; ++j) z[0][j] = s_sum[m][c + j];
    if (gated) {
#pragma unroll
      for (int j = 0; j < 8; ++j) u[0][j] = s_sum[m][8 + j];
      finish8<true, 1>(p.epi, m, 0, 1u, n0 + c, z, u);
    } else {
      finish8<false, 1>(p.epi, m, 0, 1u, n0 + c, z, u);
    }
  }
}

}  // namespace

// As many warps to a CTA as keep all CTAs resident at once (at 128 registers an
// SM holds 16 warps), 4 at least.
cudaError_t launch_linear_rows(const LinearArgs& a, const void* x, const void* w, int sms,
                               cudaStream_t s) {
  const int cols = a.epi.act == MOE_LINEAR_SWIGLU ? kRows / 2 : kRows;
  const int ctas = (a.epi.cols - 1) / cols + 1;
  const int segments = (a.K - 1) / kSegment + 1;
  int warps = kMaxWarps;
  while (warps > 4 && ctas > sms * (16 / warps)) warps /= 2;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg =
      pdl_config(dim3(ctas), dim3(32 * std::min(warps, segments)), 0, s, attr);
  return cudaLaunchKernelEx(&cfg, linear_rows_kernel, a, static_cast<const __nv_bfloat16*>(x),
                            static_cast<const __nv_bfloat16*>(w));
}

}  // namespace moe
