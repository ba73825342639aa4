// linear_epi.cuh -- the epilogue of the products in gemm_linear.cu and
// gemm_linear_rows.cu: from a row's fp32 sums z to the output,
//
//   out = act(z + bias) + residual   (SwiGLU: SiLU(z_gate) * z_up, z holding gate
//                                     then up columns)
//
// all in fp32, rounded once, and z + bias (rounded to bf16, as the gradients
// take it) where the call keeps it.  A lane has eight consecutive columns of a
// row, 16 bytes of bf16, whatever kernel the sums come from.
#pragma once

#include <cuda_bf16.h>

#include "internal.h"
#include "ptx.cuh"

namespace moe {

// With Phi the normal distribution, Phi(-|z|) and e = exp(-z^2 / 2): Phi(-|z|) / e is a smooth
// function of t = 1 / (1 + 0.35 |z|), t times a polynomial that was fitted to it over |z| <
// 14.5 (3.2e-8 relative; beyond, e is 0).  Within (8 + z^2) 2^-23 relative, and a third of
// erff's instructions; the gradient needs e anyway.
__device__ __forceinline__ float2 normal_tail(float2 z, float2& e) {
  constexpr float kP[9] = {1.396213025e-01f, 1.398635209e-01f,  1.198212728e-01f,
                           1.055525765e-01f, -2.321253717e-02f, 1.593199670e-01f,
                           -2.558392584e-01f, 1.440310478e-01f, -2.915791050e-02f};
  const float2 a = make_float2(fabsf(z.x), fabsf(z.y));
  const float2 t = inverse_fast(__ffma2_rn(both(0.35f), a, both(1.0f)));
  e = exp2_fast(__fmul2_rn(__fmul2_rn(a, a), both(-0.72134752f)));  // -log2(e) / 2
  float2 p = both(kP[8]);
#pragma unroll
  for (int i = 7; i >= 0; --i) p = __ffma2_rn(p, t, both(kP[i]));
  return __fmul2_rn(__fmul2_rn(p, t), e);
}
// z Phi(z) = max(z, 0) - |z| Phi(-|z|): within 4 2^-23 |z| of the exact one, below 0
// within (9 + z^2) 2^-23 of itself.  Infinities take the limits, inf and 0: the tail is 0
// from kTailEnd on, and what it multiplies ends there too.
constexpr float kTailEnd = 16.0f;
__device__ __forceinline__ float2 gelu(float2 z) {
  float2 e;
  const float2 h = normal_tail(z, e);
  return __ffma2_rn(
      make_float2(-fminf(fabsf(z.x), kTailEnd), -fminf(fabsf(z.y), kTailEnd)), h,
      make_float2(fmaxf(z.x, 0.0f), fmaxf(z.y, 0.0f)));
}
// 1 / (1 + e^-z) and z times it: within (8 + 1.2 |z|) 2^-23 relative, 0 below -87.3.
__device__ __forceinline__ float2 sigmoid(float2 z) {
  return inverse_fast(__fadd2_rn(both(1.0f), exp2_fast(__fmul2_rn(z, both(-1.44269504f)))));
}
// What an infinite z stands for beside a sigmoid of 0, or one less a sigmoid of 1: their product
// is the limit 0 and no NaN.
constexpr float kLargest = 3.402823466e38f;
__device__ __forceinline__ float2 silu(float2 z, float2 s) {  // s = sigmoid(z)
  return __fmul2_rn(make_float2(fmaxf(z.x, -kLargest), fmaxf(z.y, -kLargest)), s);
}
__device__ __forceinline__ float2 silu(float2 z) { return silu(z, sigmoid(z)); }

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

__device__ __forceinline__ void add_bias8(const float* b, float (&z)[8]) {
  const float4 p = __ldg(reinterpret_cast<const float4*>(b));
  const float4 q = __ldg(reinterpret_cast<const float4*>(b) + 1);
  z[0] += p.x, z[1] += p.y, z[2] += p.z, z[3] += p.w;
  z[4] += q.x, z[5] += q.y, z[6] += q.z, z[7] += q.w;
}

__device__ __forceinline__ void store_bf16x8(__nv_bfloat16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]),
                                            bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7]));
}

// Sums z (SwiGLU: gate sums z and up sums u) of columns [col, col + 8) of row
// `row` to the output.  Element by element, for rows off 16 bytes and columns
// past the last one; out of line, as its registers would cost the others.
static __device__ __noinline__ void finish8_any(const LinearEpi& e, long long row, int col,
                                                const float* z, const float* u) {
  const bool gated = e.act == MOE_LINEAR_SWIGLU;
  const long long o = row * e.cols, p = row * (gated ? 2ll * e.cols : e.cols);
  for (int i = 0; i < 8 && col + i < e.cols; ++i) {
    const int c = col + i;
    float v = z[i] + (e.bias != nullptr ? e.bias[c] : 0.0f);
    float w = 0.0f;
    if (gated) w = u[i] + (e.bias != nullptr ? e.bias[e.cols + c] : 0.0f);
    if (e.preact != nullptr) {
      e.preact[p + c] = __float2bfloat16_rn(v);
      if (gated) e.preact[p + e.cols + c] = __float2bfloat16_rn(w);
    }
    if (gated)
      v = silu(both(v)).x * w;
    else if (e.act == MOE_LINEAR_SILU)
      v = silu(both(v)).x;
    else if (e.act == MOE_LINEAR_GELU)
      v = gelu(both(v)).x;
    if (e.out_bf16) {
      if (e.residual != nullptr)
        v += __bfloat162float(static_cast<const __nv_bfloat16*>(e.residual)[o + c]);
      static_cast<__nv_bfloat16*>(e.out)[o + c] = __float2bfloat16_rn(v);
    } else {
      if (e.residual != nullptr) v += static_cast<const float*>(e.residual)[o + c];
      static_cast<float*>(e.out)[o + c] = v;
    }
  }
}

// R rows, `stride` apart from `row` on, those whose bit is set in `live`; all of them go
// through each step together, so that its loads and its branch are met once.  GATED
// (SwiGLU): u are the up sums; otherwise u is not used.
template <bool GATED, int R>
__device__ __forceinline__ void finish8(const LinearEpi& e, long long row, int stride,
                                        unsigned live, int col, float (&z)[R][8],
                                        float (&u)[GATED ? R : 1][8]) {
  if (col >= e.cols) return;
  if (!e.wide) {
#pragma unroll 1
    for (int r = 0; r < R; ++r) {
      float zs[8], us[8];  // copies, so that the others stay in registers
#pragma unroll
      for (int s = 0; s < R; ++s) {
        if (s != r) continue;
#pragma unroll
        for (int i = 0; i < 8; ++i) zs[i] = z[s][i], us[i] = u[GATED ? s : 0][i];
      }
      if ((live >> r) & 1u) finish8_any(e, row + r * stride, col, zs, us);
    }
    return;
  }
  const long long o = row * e.cols + col;
  const long long pitch = static_cast<long long>(stride) * e.cols;
  // the residual's words leave before the arithmetic
  uint4 r0[R], r1[R];
  if (e.residual != nullptr) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      r0[r] = r1[r] = make_uint4(0u, 0u, 0u, 0u);
      if (!((live >> r) & 1u)) continue;
      if (e.out_bf16) {
        r0[r] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(e.residual) + o +
                                                r * pitch);
      } else {
        const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(e.residual) + o +
                                                        r * pitch);
        r0[r] = q[0];
        r1[r] = q[1];
      }
    }
  }
  if (e.bias != nullptr) {
    float b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = 0.0f;
    add_bias8(e.bias + col, b);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < 8; ++i) z[r][i] += b[i];
    if constexpr (GATED) {
#pragma unroll
      for (int i = 0; i < 8; ++i) b[i] = 0.0f;
      add_bias8(e.bias + e.cols + col, b);
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < 8; ++i) u[r][i] += b[i];
    }
  }
  if (e.preact != nullptr) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (!((live >> r) & 1u)) continue;
      __nv_bfloat16* p = e.preact + (row + r * stride) * (GATED ? 2ll * e.cols : e.cols) + col;
      store_bf16x8(p, z[r]);
      if constexpr (GATED) store_bf16x8(p + e.cols, u[r]);
    }
  }
  if constexpr (GATED) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const float2 y = __fmul2_rn(silu(make_float2(z[r][i], z[r][i + 1])),
                                    make_float2(u[r][i], u[r][i + 1]));
        z[r][i] = y.x, z[r][i + 1] = y.y;
      }
  } else if (e.act == MOE_LINEAR_SILU) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const float2 y = silu(make_float2(z[r][i], z[r][i + 1]));
        z[r][i] = y.x, z[r][i + 1] = y.y;
      }
  } else if (e.act == MOE_LINEAR_GELU) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const float2 y = gelu(make_float2(z[r][i], z[r][i + 1]));
        z[r][i] = y.x, z[r][i + 1] = y.y;
      }
  }
  if (e.out_bf16) {
    if (e.residual != nullptr) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const uint32_t w[4] = {r0[r].x, r0[r].y, r0[r].z, r0[r].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          z[r][2 * i] += __uint_as_float(w[i] << 16);
          z[r][2 * i + 1] += __uint_as_float(w[i] & 0xffff0000u);
        }
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
      if ((live >> r) & 1u)
        store_bf16x8(static_cast<__nv_bfloat16*>(e.out) + o + r * pitch, z[r]);
  } else {
    if (e.residual != nullptr) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const uint32_t w[8] = {r0[r].x, r0[r].y, r0[r].z, r0[r].w,
                               r1[r].x, r1[r].y, r1[r].z, r1[r].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) z[r][i] += __uint_as_float(w[i]);
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (!((live >> r) & 1u)) continue;
      float4* p = reinterpret_cast<float4*>(static_cast<float*>(e.out) + o + r * pitch);
      p[0] = make_float4(z[r][0], z[r][1], z[r][2], z[r][3]);
      p[1] = make_float4(z[r][4], z[r][5], z[r][6], z[r][7]);
    }
  }
}

}  // namespace moe
