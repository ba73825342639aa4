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
// One pass: a team of lanes owns a block and keeps it in registers between
// the maximum and the codes.  Bound by HBM for fp32, and for bf16, half the
// bytes for the same arithmetic, close to its instructions: teams of 8 lanes
// with 16 columns each there (two loads and one store of 16 bytes, one
// division per 16 columns), 16 lanes with 8 columns otherwise.  T=8192 H=7168
// bf16: 29.3 us, 6080 GB/s.
#include <cuda_bf16.h>

#include <algorithm>

#include "internal.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kBlock = 128;
constexpr float kAmaxFloor = 7.8886090522101181e-31f;  // 2^-100

// SiLU by the fast exponential and division, as in the GEMMs' epilogues.  The
// product is within 3e-7 of the 64-bit one for gates down to -16 (the same
// formula in IEEE operations: 2.5e-7), 4e-6 at -80, where the exponent's
// rounding grows with the gate, and 0 below -87.3, where SiLU is under 1e-36.
// Of 33.6 million codes (T=16411 I=2048, normal gates) 37 miss the exact one
// either way.  More exact forms cost the kernel its rate (T=16411 I=2048 bf16,
// 26.7 us): the exponent's rounding made good 29.8 to 30.9, expf 31.4, expf of
// -|g| 34.0, expf and an IEEE division 40.0.
__device__ __forceinline__ float silu_mul(float g, float u) {
  return __fdividef(g, 1.0f + __expf(-g)) * u;
}

// bf16 pairs of 16-byte words as fp32.
template <int N>
__device__ __forceinline__ void bf16_words(const uint4 (&q)[N], float (&v)[8 * N]) {
#pragma unroll
  for (int h = 0; h < N; ++h) {
    const uint32_t w[4] = {q[h].x, q[h].y, q[h].z, q[h].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[8 * h + 2 * i] = __uint_as_float(w[i] << 16);
      v[8 * h + 2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

// Columns of a lane: COLS consecutive ones (WIDE, 16-byte loads; rows end on a
// multiple of COLS), or every (128 / COLS)th one with a bounds check.
template <typename T, bool WIDE, int COLS>
__device__ __forceinline__ void load_cols(const T* __restrict__ row, int c0, int lane, int H,
                                          float (&v)[COLS]) {
  if constexpr (!WIDE) {
#pragma unroll
    for (int i = 0; i < COLS; ++i) {
      const int c = c0 + lane + kBlock / COLS * i;
      v[i] = c < H ? static_cast<float>(row[c]) : 0.0f;
    }
  } else {
    const int c = c0 + COLS * lane;
    if (c >= H) {
#pragma unroll
      for (int i = 0; i < COLS; ++i) v[i] = 0.0f;
    } else if constexpr (sizeof(T) == 2) {
      uint4 q[COLS / 8];
#pragma unroll
      for (int h = 0; h < COLS / 8; ++h) q[h] = reinterpret_cast<const uint4*>(row + c)[h];
      bf16_words(q, v);
    } else {
#pragma unroll
      for (int h = 0; h < COLS / 4; ++h) {
        const float4 p = reinterpret_cast<const float4*>(row + c)[h];
        v[4 * h] = p.x;
        v[4 * h + 1] = p.y;
        v[4 * h + 2] = p.z;
        v[4 * h + 3] = p.w;
      }
    }
  }
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t h;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(hi), "f"(lo));
  return h;
}

// The block's maximum over the lanes of its team, at least the floor.
template <int COLS>
__device__ __forceinline__ float block_max(const float (&v)[COLS], unsigned team) {
  float m = kAmaxFloor;
#pragma unroll
  for (int i = 0; i < COLS; ++i) m = fmaxf(m, fabsf(v[i]));
#pragma unroll
  for (int d = kBlock / COLS / 2; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(team, m, d));
  return m;
}

// The codes of COLS consecutive columns, one store.
template <int COLS>
__device__ __forceinline__ void store_codes(const float (&v)[COLS], float r, uint8_t* q) {
  uint32_t p[COLS / 4];
#pragma unroll
  for (int i = 0; i < COLS / 4; ++i)
    p[i] = e4m3x2(v[4 * i] * r, v[4 * i + 1] * r) |
           (e4m3x2(v[4 * i + 2] * r, v[4 * i + 3] * r) << 16);
  if constexpr (COLS == 16)
    *reinterpret_cast<uint4*>(q) = make_uint4(p[0], p[1], p[2], p[3]);
  else
    *reinterpret_cast<uint2*>(q) = make_uint2(p[0], p[1]);
}

template <typename T, bool GATED, bool WIDE, int COLS>
__global__ void __launch_bounds__(kThreads)
    quantize_block_kernel(const T* __restrict__ x, unsigned blocks, int H, unsigned nb,
                          uint8_t* __restrict__ xq, float* __restrict__ scale) {
  constexpr int LANES = kBlock / COLS;
  constexpr unsigned kTeams = kThreads / LANES;
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & (LANES - 1);
  const unsigned team = ((1u << LANES) - 1u) << (threadIdx.x & (32 - LANES));
  const unsigned j = blockIdx.x * kTeams + threadIdx.x / LANES;
  if (j >= blocks) return;
  const unsigned t = j / nb;
  const int c0 = static_cast<int>(j - t * nb) * kBlock;
  const T* row = x + static_cast<long long>(t) * (GATED ? 2ll * H : H);
  float v[COLS];
  load_cols<T, WIDE, COLS>(row, c0, lane, H, v);
  if constexpr (GATED) {
    float u[COLS];
    load_cols<T, WIDE, COLS>(row + H, c0, lane, H, u);
#pragma unroll
    for (int i = 0; i < COLS; ++i) v[i] = silu_mul(v[i], u[i]);
  }
  const float m = block_max<COLS>(v, team);
  const float r = __fdiv_rn(448.0f, m);
  if (lane == 0) scale[j] = __fdiv_rn(m, 448.0f);
  uint8_t* q = xq + static_cast<long long>(t) * H;
  if constexpr (WIDE) {
    if (c0 + COLS * lane < H) store_codes<COLS>(v, r, q + c0 + COLS * lane);
  } else {
#pragma unroll
    for (int i = 0; i < COLS; ++i) {
      const int c = c0 + lane + LANES * i;
      if (c < H) q[c] = static_cast<uint8_t>(e4m3x2(v[i] * r, 0.0f));
    }
  }
}

// Gated bf16 rows of a multiple of 16 columns: 8 lanes of 16 columns walk
// blocks a grid apart with the next one's words in flight while they encode
// one, four CTAs per SM (T=16411 I=2048: 26.9 us against 33.0 with a block per
// team, whose loads wait for other CTAs' exponentials and divisions; T=4096:
// 8.7 against 9.4).  The other inputs have too little arithmetic for it: bf16
// rows of T=8192 H=7168 took 31.9 us this way and 29.7 with a block per team,
// gated fp32 46.5 and 44.9.
__global__ void __launch_bounds__(kThreads)
    quantize_gated_kernel(const __nv_bfloat16* __restrict__ x, unsigned blocks, int H, unsigned nb,
                          uint8_t* __restrict__ xq, float* __restrict__ scale) {
  constexpr int COLS = 16, LANES = kBlock / COLS;
  constexpr unsigned kTeams = kThreads / LANES;
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & (LANES - 1);
  const unsigned team = ((1u << LANES) - 1u) << (threadIdx.x & (32 - LANES));
  const unsigned step = gridDim.x * kTeams;
  uint4 g[2], u[2];
  auto load = [&](unsigned j) {
    if (j >= blocks) return;
    const unsigned t = j / nb;
    const int c = static_cast<int>(j - t * nb) * kBlock + COLS * lane;
    if (c >= H) return;
    const __nv_bfloat16* row = x + static_cast<long long>(t) * 2 * H + c;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      g[i] = reinterpret_cast<const uint4*>(row)[i];
      u[i] = reinterpret_cast<const uint4*>(row + H)[i];
    }
  };
  unsigned j = blockIdx.x * kTeams + threadIdx.x / LANES;
  load(j);
  for (; j < blocks; j += step) {
    const unsigned t = j / nb;
    const int c = static_cast<int>(j - t * nb) * kBlock + COLS * lane;
    float v[COLS], w[COLS];
    bf16_words(g, v);
    bf16_words(u, w);
    load(j + step);
#pragma unroll
    for (int i = 0; i < COLS; ++i) v[i] = silu_mul(v[i], w[i]);
    if (c >= H) {  // the last block's lanes past the row
#pragma unroll
      for (int i = 0; i < COLS; ++i) v[i] = 0.0f;
    }
    const float m = block_max<COLS>(v, team);
    const float r = __fdiv_rn(448.0f, m);
    if (lane == 0) scale[j] = __fdiv_rn(m, 448.0f);
    if (c < H) store_codes<COLS>(v, r, xq + static_cast<long long>(t) * H + c);
  }
}

template <typename T, bool GATED, bool WIDE, int COLS>
cudaError_t launch_cols(const T* x, int rows, int H, uint8_t* xq, float* scale, cudaStream_t s) {
  const unsigned nb = static_cast<unsigned>((H + kBlock - 1) / kBlock);
  const unsigned blocks = static_cast<unsigned>(rows) * nb;  // the caller checks that it fits
  const unsigned teams = kThreads / (kBlock / COLS);
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg =
      pdl_config(dim3(blocks / teams + (blocks % teams != 0)), dim3(kThreads), 0, s, attr);
  return cudaLaunchKernelEx(&cfg, quantize_block_kernel<T, GATED, WIDE, COLS>, x, blocks, H, nb,
                            xq, scale);
}

cudaError_t launch_gated(const __nv_bfloat16* x, int rows, int H, uint8_t* xq, float* scale,
                         cudaStream_t s) {
  const unsigned nb = static_cast<unsigned>((H + kBlock - 1) / kBlock);
  const unsigned blocks = static_cast<unsigned>(rows) * nb;
  const unsigned teams = kThreads / 8;
  const unsigned ctas = blocks / teams + (blocks % teams != 0);
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg =
      pdl_config(dim3(std::min(ctas, 4u * device_sm_count())), dim3(kThreads), 0, s, attr);
  return cudaLaunchKernelEx(&cfg, quantize_gated_kernel, x, blocks, H, nb, xq, scale);
}

template <typename T, bool GATED>
cudaError_t launch_as(const void* x, int rows, int H, uint8_t* xq, float* scale, cudaStream_t s) {
  auto aligned = [&](int cols, unsigned out) {
    return H % cols == 0 && (reinterpret_cast<uintptr_t>(x) & 15u) == 0 &&
           (reinterpret_cast<uintptr_t>(xq) & (out - 1)) == 0;
  };
  const T* xt = static_cast<const T*>(x);
  if constexpr (sizeof(T) == 2) {
    if (GATED && aligned(16, 16)) return launch_gated(xt, rows, H, xq, scale, s);
    if constexpr (!GATED)
      if (aligned(16, 16)) return launch_cols<T, false, true, 16>(xt, rows, H, xq, scale, s);
  }
  if (aligned(8, 8)) return launch_cols<T, GATED, true, 8>(xt, rows, H, xq, scale, s);
  return launch_cols<T, GATED, false, 8>(xt, rows, H, xq, scale, s);
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
