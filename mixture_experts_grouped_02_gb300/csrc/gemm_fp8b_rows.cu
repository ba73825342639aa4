// gemm_fp8b_rows.cu -- the plain product of gemm_fp8b.cu for at most eight rows
// of a (decode): streaming the weights once is all there is to do, and what
// counts is how early the loads leave and how few steps follow them.
//
//   out[m, n] = sum_b sa[m, b] * sb[n / 128, b] * sum_{k in block b} a[m, k] * w[n, k]
//
// A CTA owns 16 weight rows and all of K; its warps take the scale blocks in
// turn and add their partial sums through shared memory, in warp order.  The
// products are mma.sync m16n8k32 with the weights as the 16-row operand and
// the rows of a as the 8-column one: no shared memory or TMEM stands between a
// load and its MMA.  The K positions inside a scale block are dealt to the
// fragments so that a lane's four MMAs take 32 consecutive bytes of a row
// (both operands the same way, so the sum is the same).  mma.sync runs far
// below the tcgen05 rate, which does not matter here: a warp issues four MMAs
// for every 2 KB of weights.  Row m of a fills column m of the MMA, so a NaN
// or an infinite scale stays in its row.
//
// Bound by latency: a launch, and one trip to HBM per warp while 16 warps of
// four blocks cover K, or two in turn with 8 warps to a CTA, as a warp's loads
// wait in registers (four blocks, at the cap of 128 registers, where it spills 16
// bytes).  Measured (us, weights from HBM; the best tcgen05 form in brackets):
// one row, 7168 x 2048 5.9 (7.2), 576 x 7168 4.7 (6.7), 2048 x 7168 6.2 (8.8),
// 4096 x 7168 9.2 (11.5), 47 % of the copy rate; eight rows, 7168 x 2048 6.2
// (6.9), 4096 x 7168 10.0 (11.3).  With the weights in L2 one row takes 4.6 us for
// 7168 x 2048 and 7.8 for 4096 x 7168.  Sixteen rows, in two columns of MMAs,
// gained 15 % at best and lost on others; lists of small blocks (16 rows, 64
// blocks of N=4096 K=7168) took 143 against 119.
#include <cuda_bf16.h>

#include <algorithm>

#include "internal.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kRows = 16;     // weight rows of a CTA
constexpr int kTokens = 8;    // rows of a
constexpr int kMaxWarps = 16;
constexpr int kInFlight = 4;  // scale blocks a warp loads at once

__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The 32 bytes at byte k of a row of K (a multiple of 16), zero past K.
__device__ __forceinline__ void load32(const uint8_t* row, int k, int K, uint4 (&v)[2]) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
    v[h] = k + 16 * h < K ? __ldg(reinterpret_cast<const uint4*>(row + k + 16 * h))
                          : make_uint4(0u, 0u, 0u, 0u);
}

__global__ void __launch_bounds__(kMaxWarps * 32)
    fp8b_rows_kernel(const Fp8bArgs p, const uint8_t* __restrict__ a,
                     const uint8_t* __restrict__ w) {
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
  const int n0 = blockIdx.x * kRows;
  const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  // rows past N read the last one and are not stored
  const uint8_t* w0 = w + static_cast<long long>(min(n0 + g, p.N - 1)) * p.K;
  const uint8_t* w1 = w + static_cast<long long>(min(n0 + g + 8, p.N - 1)) * p.K;
  const uint8_t* row = a + static_cast<long long>(min(g, p.M - 1)) * p.K;
  const float* sb = p.w_scale + static_cast<long long>(n0 / 128) * p.k_tiles;
  float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};

  for (int kb = warp; kb < p.k_tiles; kb += U * warps) {
    uint4 x0[U][2], x1[U][2], y[U][2];
    float s[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int blk = kb + u * warps;
      const int k = blk < p.k_tiles ? blk * 128 + 32 * t : p.K;
      load32(w0, k, p.K, x0[u]);
      load32(w1, k, p.K, x1[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int blk = kb + u * warps;
      const bool in = blk < p.k_tiles;
      load32(row, in && g < p.M ? blk * 128 + 32 * t : p.K, p.K, y[u]);
      const float ws = in ? __ldg(sb + blk) : 0.0f;
#pragma unroll
      for (int h = 0; h < 2; ++h)  // the two rows of a whose sums this lane holds
        s[u][h] = in && 2 * t + h < p.M
                      ? __ldg(p.a_scale + static_cast<long long>(2 * t + h) * p.k_tiles + blk) * ws
                      : 0.0f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (kb + u * warps >= p.k_tiles) break;
      const uint32_t a0[8] = {x0[u][0].x, x0[u][0].y, x0[u][0].z, x0[u][0].w,
                              x0[u][1].x, x0[u][1].y, x0[u][1].z, x0[u][1].w};
      const uint32_t a1[8] = {x1[u][0].x, x1[u][0].y, x1[u][0].z, x1[u][0].w,
                              x1[u][1].x, x1[u][1].y, x1[u][1].z, x1[u][1].w};
      const uint32_t b[8] = {y[u][0].x, y[u][0].y, y[u][0].z, y[u][0].w,
                             y[u][1].x, y[u][1].y, y[u][1].z, y[u][1].w};
      float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int q = 0; q < 4; ++q)
        mma_e4m3(d, a0[2 * q], a1[2 * q], a0[2 * q + 1], a1[2 * q + 1], b[2 * q], b[2 * q + 1]);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = fmaf(s[u][i & 1], d[i], acc[i]);
    }
  }
  s_part[warp][2 * t][g] = acc[0];
  s_part[warp][2 * t + 1][g] = acc[1];
  s_part[warp][2 * t][g + 8] = acc[2];
  s_part[warp][2 * t + 1][g + 8] = acc[3];
  if (threadIdx.x == 0) s_stop = stop;
  __syncthreads();
  if (s_stop != 0) return;
  for (int i = threadIdx.x; i < p.M * kRows; i += blockDim.x) {
    const int m = i / kRows, c = i % kRows;
    if (n0 + c >= p.N) continue;
    float sum = 0.0f;
    for (int v = 0; v < warps; ++v) sum += s_part[v][m][c];
    const long long o = static_cast<long long>(m) * p.N + n0 + c;
    if (p.out_bf16)
      static_cast<__nv_bfloat16*>(p.out)[o] = __float2bfloat16_rn(sum);
    else
      static_cast<float*>(p.out)[o] = sum;
  }
}

}  // namespace

// As many warps to a CTA as keep all CTAs resident at once (at 128 registers
// an SM holds 16 warps), 4 at least: with the weights in L2 one row of 4096 x
// 7168 takes 7.8 us with 8 warps (256 CTAs) and 9.5 with 16, of 2048 x 7168 4.8
// with 16 and 5.3 with 8.
cudaError_t launch_fp8b_rows(const Fp8bArgs& a, const uint8_t* x, const uint8_t* w, int sms,
                             cudaStream_t s) {
  const int ctas = (a.N + kRows - 1) / kRows;
  int warps = kMaxWarps;
  while (warps > 4 && ctas > sms * (16 / warps)) warps /= 2;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg =
      pdl_config(dim3(ctas), dim3(32 * std::min(warps, a.k_tiles)), 0, s, attr);
  return cudaLaunchKernelEx(&cfg, fp8b_rows_kernel, a, x, w);
}

}  // namespace moe
