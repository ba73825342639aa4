// quant_block.cu -- rows to e4m3 codes with one fp32 scale per 128 columns,
// of the rows themselves or of SiLU(gate) * up.
//
// For columns [128 b, 128 b + 128) of a row of v (the last block may be
// shorter): m = max(max |v|, 2^-100), scale = m / 448, code = e4m3(v * (448 /
// m)), all in fp32 with IEEE rounding, the code rounded to nearest even and
// saturated.  The floor 2^-100 keeps 448 / m finite and the scale normal, so
// an all-zero or subnormal block gives exact zeros or codes of its own scale
// instead of 0 * inf.  A NaN becomes the NaN code; an infinity makes the
// block's scale infinite and the block NaN.  Source: "MOE Bmm1 Fused Gather",
// pack_e4m3x2 (the conversion instruction), with the scale per 128 columns
// that DeepSeek-V3's fp8 weights go with.
//
// Gated: v = gate / (1 + e^-gate) * up, the row holding gate then up.
//
// One pass: 16 lanes own a block, 8 columns each, kept in registers between
// the maximum and the codes.  Bound by HBM.
#include <cuda_bf16.h>

#include <algorithm>

#include "internal.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kLanes = 16;                       // lanes of a block
constexpr int kCols = 8;                         // columns of a lane
constexpr int kBlock = kLanes * kCols;           // 128
constexpr int kTeams = kThreads / kLanes;
constexpr float kAmaxFloor = 7.8886090522101181e-31f;  // 2^-100

__device__ __forceinline__ float silu_mul(float g, float u) {
  return __fdividef(g, 1.0f + __expf(-g)) * u;
}

// Columns of this lane: 8 consecutive ones (WIDE, 16-byte loads), or every
// 16th one with a bounds check.
template <typename T, bool WIDE>
__device__ __forceinline__ void load_cols(const T* __restrict__ row, int c0, int lane, int H,
                                          float (&v)[kCols]) {
  if constexpr (!WIDE) {
#pragma unroll
    for (int i = 0; i < kCols; ++i) {
      const int c = c0 + lane + kLanes * i;
      v[i] = c < H ? static_cast<float>(row[c]) : 0.0f;
    }
  } else {
    const int c = c0 + kCols * lane;
    if (c >= H) {  // H is a multiple of 8
#pragma unroll
      for (int i = 0; i < kCols; ++i) v[i] = 0.0f;
    } else if constexpr (sizeof(T) == 2) {
      const uint4 q = *reinterpret_cast<const uint4*>(row + c);
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    } else {
      const float4 p = reinterpret_cast<const float4*>(row + c)[0];
      const float4 q = reinterpret_cast<const float4*>(row + c)[1];
      v[0] = p.x, v[1] = p.y, v[2] = p.z, v[3] = p.w;
      v[4] = q.x, v[5] = q.y, v[6] = q.z, v[7] = q.w;
    }
  }
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t h;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(hi), "f"(lo));
  return h;
}

template <typename T, bool GATED, bool WIDE>
__global__ void __launch_bounds__(kThreads)
    quantize_block_kernel(const T* __restrict__ x, long long blocks, int H, int nb,
                          uint8_t* __restrict__ xq, float* __restrict__ scale) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & (kLanes - 1);
  const unsigned half = 0xffffu << (threadIdx.x & 16);
  for (long long j = static_cast<long long>(blockIdx.x) * kTeams + threadIdx.x / kLanes;
       j < blocks; j += static_cast<long long>(gridDim.x) * kTeams) {
    const long long t = j / nb;
    const int c0 = static_cast<int>(j - t * nb) * kBlock;
    const T* row = x + t * (GATED ? 2ll * H : H);
    float v[kCols];
    load_cols<T, WIDE>(row, c0, lane, H, v);
    if constexpr (GATED) {
      float u[kCols];
      load_cols<T, WIDE>(row + H, c0, lane, H, u);
#pragma unroll
      for (int i = 0; i < kCols; ++i) v[i] = silu_mul(v[i], u[i]);
    }
    float m = kAmaxFloor;
#pragma unroll
    for (int i = 0; i < kCols; ++i) m = fmaxf(m, fabsf(v[i]));
#pragma unroll
    for (int d = kLanes / 2; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(half, m, d));
    const float r = __fdiv_rn(448.0f, m);
    if (lane == 0) scale[j] = __fdiv_rn(m, 448.0f);
    uint8_t* q = xq + t * H;
    if constexpr (WIDE) {
      if (c0 + kCols * lane < H) {
        const uint32_t a = e4m3x2(v[0] * r, v[1] * r) | (e4m3x2(v[2] * r, v[3] * r) << 16);
        const uint32_t b = e4m3x2(v[4] * r, v[5] * r) | (e4m3x2(v[6] * r, v[7] * r) << 16);
        *reinterpret_cast<uint2*>(q + c0 + kCols * lane) = make_uint2(a, b);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kCols; ++i) {
        const int c = c0 + lane + kLanes * i;
        if (c < H) q[c] = static_cast<uint8_t>(e4m3x2(v[i] * r, 0.0f));
      }
    }
  }
}

template <typename T, bool GATED>
cudaError_t launch_as(const void* x, int T_, int H, uint8_t* xq, float* scale, cudaStream_t s) {
  const int nb = (H + kBlock - 1) / kBlock;
  const long long blocks = static_cast<long long>(T_) * nb;
  const unsigned grid = static_cast<unsigned>(
      std::min<long long>((blocks + kTeams - 1) / kTeams, 0x7fffffffll));
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = pdl_config(dim3(grid), dim3(kThreads), 0, s, attr);
  const bool wide = H % kCols == 0 && (reinterpret_cast<uintptr_t>(x) & 15u) == 0 &&
                    (reinterpret_cast<uintptr_t>(xq) & 7u) == 0;
  const T* xt = static_cast<const T*>(x);
  if (wide)
    return cudaLaunchKernelEx(&cfg, quantize_block_kernel<T, GATED, true>, xt, blocks, H, nb, xq,
                              scale);
  return cudaLaunchKernelEx(&cfg, quantize_block_kernel<T, GATED, false>, xt, blocks, H, nb, xq,
                            scale);
}

}  // namespace

cudaError_t launch_quantize_block(const void* x, int x_dtype, int T, int H, int gated,
                                  uint8_t* xq, float* scale, cudaStream_t s) {
  if (x_dtype == MOE_BF16)
    return gated ? launch_as<__nv_bfloat16, true>(x, T, H, xq, scale, s)
                 : launch_as<__nv_bfloat16, false>(x, T, H, xq, scale, s);
  return gated ? launch_as<float, true>(x, T, H, xq, scale, s)
               : launch_as<float, false>(x, T, H, xq, scale, s);
}

}  // namespace moe
