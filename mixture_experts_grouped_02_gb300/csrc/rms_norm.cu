// rms_norm.cu -- RMS norm of rows with the residual's addition, the result as
// rows, as e4m3 codes with a scale per 128 columns, or both; and its gradients.
//
//   s = x + residual (fp32), rstd = 1 / sqrt(mean(s^2) + eps), y = s * rstd * w
//   sum = s rounded, out = y rounded, codes of y as in quant_block.cu
//
// Everything between the inputs and the outputs is fp32: the norm and the codes
// are of the unrounded sum, so that adding the residual here costs no rounding
// that a norm of the stored sum would have.  Sums of squares run along a
// thread's columns, then across the lanes and warps of the row's team in a
// fixed order.
//
// Gradients, with h the stored sum (or x), xhat = h * rstd and g = dy * w:
//   dx = rstd * (g - xhat * mean(g * xhat)) + dsum,   dw = sum over rows of dy * xhat
// dw's sum over rows: every team adds its rows in order in fp32 registers, the
// CTAs' parts go to a scratch and a second kernel adds those, in order as well.
//
// Both directions are bound by HBM: a row is read once, held by its team between the sum
// and its use, and the registers and shared memory per thread are set by how many bytes
// the SM's teams then have on their way.  GB300, operands from HBM, us (copy rate 6.8
// TB/s: us): T=8192 H=7168 bf16 rows 37.0 (34.5), with a residual and its sum 69.3 (69.1),
// their codes as well 78.1 (77.7); fp32 rows 71.4 (69.1), with a residual 136 (138.2).
// Gradients with the sum's: T=8192 H=4096 bf16 49.3 (39.5), H=7168 79 (69.1), fp32 148
// (138.2).
#include <cuda_bf16.h>

#include <algorithm>

#include "internal.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kVec = 8;  // columns of a lane: 16 bytes of bf16
constexpr int kBlock = 128;
constexpr float kAmaxFloor = 7.8886090522101181e-31f;  // 2^-100, as in quant_block.cu
constexpr int kMaxThreads = 1024;
// Registers of a gradient's thread that its launch bounds leave: two fp32 vectors, or two
// of single elements, which are held, spill at 64 (fp32, a CTA to a row, T=8192 H=7168:
// 145 us against 150 with one vector and 64; a warp to a row, T=32768 H=512: 44 against
// 53).
constexpr int grad_regs(int es, int vpt, bool wide) {
  return vpt == 2 && (es == 4 || !wide) ? 128 : 64;
}
constexpr int kWarpRows = 8;       // rows (warps) of a CTA where a warp takes a row

// ------------------------------------------------------------- eight columns
// A warp covers 256 columns at a time, eight to a lane.  WIDE (H % 8 == 0, rows on 16
// bytes): eight consecutive ones, which 16-byte words hold.  Otherwise every 32nd,
// so that the warp's accesses of single elements touch one line each (with eight
// consecutive ones T=8192 H=2883 bf16 took 153 us for the norm of a sum).  `c` is the
// lane's first column of the WIDE kind; column(c, i) its i-th one.

template <bool WIDE>
__device__ __forceinline__ long long column(long long c, int i) {
  const int lane = threadIdx.x & 31;
  return WIDE ? c + i : c - (kVec - 1) * lane + 32 * i;
}

// 16-byte words as fp32 values.
template <typename T>
__device__ __forceinline__ void word_values(const uint4 (&q)[sizeof(T) / 2], float (&v)[kVec]) {
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) {
    const uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (sizeof(T) == 2) {
        v[2 * j] = __uint_as_float(w[j] << 16);
        v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
      } else {
        v[4 * i + j] = __uint_as_float(w[j]);
      }
    }
  }
}

// The same as pairs.
template <typename T>
__device__ __forceinline__ void word_pairs(const uint4 (&q)[sizeof(T) / 2],
                                           float2 (&v)[kVec / 2]) {
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) {
    if constexpr (sizeof(T) == 2) {
      const uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        v[j] = make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u));
    } else {
      v[2 * i] = make_float2(__uint_as_float(q[i].x), __uint_as_float(q[i].y));
      v[2 * i + 1] = make_float2(__uint_as_float(q[i].z), __uint_as_float(q[i].w));
    }
  }
}

// A lane's columns of a row, zero past H.
template <typename T, bool WIDE>
__device__ __forceinline__ void load8(const T* row, long long c, int H, float (&v)[kVec]) {
  if constexpr (WIDE) {
    uint4 q[sizeof(T) / 2];
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i)
      q[i] = c < H ? reinterpret_cast<const uint4*>(row + c)[i] : make_uint4(0u, 0u, 0u, 0u);
    word_values<T>(q, v);
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const long long k = column<false>(c, i);
      v[i] = k < H ? static_cast<float>(row[k]) : 0.0f;
    }
  }
}

template <typename T>
__device__ __forceinline__ T rounded(float v);
template <>
__device__ __forceinline__ float rounded<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 rounded<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

template <typename T, bool WIDE>
__device__ __forceinline__ void store8(T* row, long long c, int H,
                                       const float (&v)[kVec]) {
  if constexpr (!WIDE) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const long long k = column<false>(c, i);
      if (k < H) row[k] = rounded<T>(v[i]);
    }
  } else if (c >= H) {
  } else if constexpr (sizeof(T) == 2) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
    *reinterpret_cast<uint4*>(row + c) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    *reinterpret_cast<float4*>(row + c) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(row + c + 4) = make_float4(v[4], v[5], v[6], v[7]);
  }
}

// Weights are fp32 or bf16, whatever the rows are; their 16-byte loads need
// their own alignment, which the host checks.
template <bool WIDE>
__device__ __forceinline__ void load_w8(const void* w, int w_bf16, long long c, int H,
                                        float (&v)[kVec]) {
  if (w_bf16)
    load8<__nv_bfloat16, WIDE>(static_cast<const __nv_bfloat16*>(w), c, H, v);
  else
    load8<float, WIDE>(static_cast<const float*>(w), c, H, v);
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t h;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(hi), "f"(lo));
  return h;
}

// Codes and scales of a warp's 256 columns: 16 lanes hold a block of 128 (WIDE), or
// all lanes four columns of each of two.
template <bool WIDE>
__device__ __forceinline__ void quantize8(const float (&v)[kVec], long long c, int H,
                                          uint8_t* q, float* scale) {
  if constexpr (WIDE) {
    float m = kAmaxFloor;
#pragma unroll
    for (int i = 0; i < kVec; i += 2) m = fmaxf(fmaxf(m, fabsf(v[i])), fabsf(v[i + 1]));
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    if (c >= H) return;
    const float r = __fdiv_rn(448.0f, m);
    if (c % kBlock == 0) scale[c / kBlock] = __fdiv_rn(m, 448.0f);
    uint32_t p[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 r2 = make_float2(r, r);
      const float2 lo = __fmul2_rn(make_float2(v[4 * i], v[4 * i + 1]), r2);
      const float2 hi = __fmul2_rn(make_float2(v[4 * i + 2], v[4 * i + 3]), r2);
      p[i] = e4m3x2(lo.x, lo.y) | (e4m3x2(hi.x, hi.y) << 16);
    }
    *reinterpret_cast<uint2*>(q + c) = make_uint2(p[0], p[1]);
  } else {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      float m = kAmaxFloor;
#pragma unroll
      for (int i = 4 * b; i < 4 * b + 4; ++i) m = fmaxf(m, fabsf(v[i]));
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
      const float r = __fdiv_rn(448.0f, m);
      const long long first = column<false>(c, 4 * b);
      if (first % kBlock == 0 && first < H) scale[first / kBlock] = __fdiv_rn(m, 448.0f);
#pragma unroll
      for (int i = 4 * b; i < 4 * b + 4; ++i) {
        const long long k = column<false>(c, i);
        if (k < H) q[k] = static_cast<uint8_t>(e4m3x2(v[i] * r, 0.0f));
      }
    }
  }
}

// The sum of `v` over the team of a row: LANES lanes of a warp, or (0) the CTA (one
// barrier; `s` alternates between two buffers of 32 from call to call).
template <int LANES>
__device__ __forceinline__ float team_sum(float v, float* s) {
#pragma unroll
  for (int d = LANES == 16 ? 8 : 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  if constexpr (LANES == 0) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0) s[warp] = v;
    __syncthreads();
    v = lane < warps ? s[lane] : 0.0f;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  }
  return v;
}

// ------------------------------------------------------------ rows in flight
// A thread's 16-byte words of the rows it will work on next, fetched by cp.async to
// slots of shared memory that no other thread uses: no barrier, and no registers
// held while HBM answers.  `depth` rows are in flight or being worked on, each a
// group of copies; rows that are not wide are loaded when their turn comes.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 shared16(uint32_t src) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(src)
               : "memory");
  return v;
}
__device__ __forceinline__ void copies_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// Waits until at most depth - 1 groups are in flight.
__device__ __forceinline__ void copies_wait(int depth) {
  switch (depth) {
    case 2:
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      break;
    case 3:
      asm volatile("cp.async.wait_group 2;" ::: "memory");
      break;
    case 4:
      asm volatile("cp.async.wait_group 3;" ::: "memory");
      break;
    default:
      asm volatile("cp.async.wait_group 0;" ::: "memory");
  }
}

// The rows t, t + step, ... of up to ARRAYS tensors (null ones are left out).
template <typename T, bool WIDE, int ARRAYS, int VPT>
struct Ring {
  const T* base[ARRAYS];
  uint32_t slots, pitch;  // shared addresses: this thread's first word, to its next one
  uint32_t head = 0;      // bytes from slots to the slot of the row being worked on
  int depth, H, rows, c, stride;  // stride: columns from a vector to the thread's next
  long long step;         // rows

  __device__ __forceinline__ Ring(const void* const (&tensors)[ARRAYS], uint4* smem, int depth_,
                                  int team, int member, int H_, int rows_, long long step_)
      : slots(smem_u32(smem + threadIdx.x)),
        pitch(blockDim.x * 16),
        depth(depth_),
        H(H_),
        rows(rows_),
        c(member * kVec),
        stride(team * kVec),
        step(step_) {
#pragma unroll
    for (int k = 0; k < ARRAYS; ++k)
      base[k] = static_cast<const T*>(tensors[k]);
  }
  __device__ __forceinline__ static constexpr uint32_t word(int k, int j, int w) {
    return (k * VPT + j) * (sizeof(T) / 2) + w;
  }
  // First column of a thread's word w of vector j.  fp32: the words of a warp's 256
  // columns lie one behind the other, the second ones after the first (two words of a
  // thread side by side would have every access read half of its sectors).
  __device__ __forceinline__ int column_of(int j, int w) const {
    return c + j * stride + (sizeof(T) == 4 ? 128 * w - 4 * static_cast<int>(threadIdx.x & 31) : 0);
  }
  __device__ __forceinline__ void fetch(long long row, uint32_t to) {
    if (row < rows) {
      const long long at = row * H;
#pragma unroll
      for (int k = 0; k < ARRAYS; ++k) {
        if (base[k] == nullptr) continue;
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
          for (int w = 0; w < static_cast<int>(sizeof(T) / 2); ++w)
            if (column_of(j, w) < H)
              copy16(slots + to + word(k, j, w) * pitch, base[k] + at + column_of(j, w));
      }
    }
    copies_commit();
  }
  // The first rows on their way.
  __device__ __forceinline__ void start(long long row) {
    if constexpr (WIDE)
      for (int s = 0; s < depth; ++s) fetch(row + s * step, s * word(ARRAYS, 0, 0) * pitch);
  }
  __device__ __forceinline__ void wait() {
    if constexpr (WIDE) copies_wait(depth);
  }
  // Vector j of tensor k of the row being worked on, as pairs.
  __device__ __forceinline__ void get(long long row, int k, int j, float2 (&v)[kVec / 2]) const {
    if constexpr (WIDE) {
      uint4 q[sizeof(T) / 2];
#pragma unroll
      for (int w = 0; w < static_cast<int>(sizeof(T) / 2); ++w)
        q[w] = shared16(slots + head + word(k, j, w) * pitch);
      word_pairs<T>(q, v);
    } else {
      float f[kVec];
      load8<T, false>(base[k] + row * H, c + j * stride, H, f);
#pragma unroll
      for (int i = 0; i < kVec / 2; ++i) v[i] = make_float2(f[2 * i], f[2 * i + 1]);
    }
  }
  // The slots past the row's end, which fetch leaves alone, as zeros.
  __device__ __forceinline__ void clear() const {
    if constexpr (WIDE) {
#pragma unroll
      for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int w = 0; w < static_cast<int>(sizeof(T) / 2); ++w) {
          if (column_of(j, w) < H) continue;
          for (int s = 0; s < depth; ++s)
#pragma unroll
            for (int k = 0; k < ARRAYS; ++k)
              asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(
                               slots + (s * word(ARRAYS, 0, 0) + word(k, j, w)) * pitch),
                           "r"(0)
                           : "memory");
        }
    }
  }
  // The thread's values v of vector j to a row of `out`, and its weights.
  template <typename O>
  __device__ __forceinline__ void put(O* out, int j, const float (&v)[kVec]) const {
    if constexpr (WIDE && sizeof(T) == 4) {
#pragma unroll
      for (int w = 0; w < 2; ++w)
        if (column_of(j, w) < H)
          *reinterpret_cast<float4*>(out + column_of(j, w)) =
              make_float4(v[4 * w], v[4 * w + 1], v[4 * w + 2], v[4 * w + 3]);
    } else {
      store8<O, WIDE>(out, c + j * stride, H, v);
    }
  }
  __device__ __forceinline__ void weights(const void* p, int p_bf16, int j, float (&v)[kVec]) const {
    if constexpr (WIDE && sizeof(T) == 4) {
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const int k = column_of(j, w);
        float4 q = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (k < H && p_bf16) {
          const uint2 b = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p) + k);
          q = make_float4(__uint_as_float(b.x << 16), __uint_as_float(b.x & 0xffff0000u),
                          __uint_as_float(b.y << 16), __uint_as_float(b.y & 0xffff0000u));
        } else if (k < H) {
          q = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + k);
        }
        v[4 * w] = q.x, v[4 * w + 1] = q.y, v[4 * w + 2] = q.z, v[4 * w + 3] = q.w;
      }
    } else {
      load_w8<WIDE>(p, p_bf16, c + j * stride, H, v);
    }
  }
  // All of this row has been read: its slot takes the row `depth` steps on.
  __device__ __forceinline__ void next(long long row) {
    if constexpr (WIDE) {
      fetch(row + depth * step, head);
      head += word(ARRAYS, 0, 0) * pitch;
      if (head == depth * word(ARRAYS, 0, 0) * pitch) head = 0;
    }
  }
};

int round_up(int n, int to) { return (n + to - 1) / to * to; }

// The most shared memory that a gradient's launch may want.
constexpr int kMostSmem = 226 * 1024;

// How rows are dealt to CTAs: `threads` of a CTA, slots for `depth` rows, CTAs in all.
struct RowForm {
  int threads, depth, ctas;
  size_t ring_bytes;
};

// An SM's shared memory goes to its resident CTAs, as many as `regs` registers a
// thread allow, up to four rows each.
RowForm row_form(int T, int es, int arrays, bool wide, bool warp_row, int vpt, int threads,
                 int regs, size_t more_smem, int sms) {
  RowForm f;
  f.threads = threads;
  const int teams = warp_row ? (T - 1) / kWarpRows + 1 : T;
  const int per_sm = std::max(1, std::min(2048, 65536 / regs) / threads);
  const size_t row = static_cast<size_t>(threads) * vpt * kVec * es * arrays;
  const size_t share = 220 * 1024 / per_sm - 1024 - more_smem;
  f.depth = wide ? static_cast<int>(std::max<size_t>(1, std::min<size_t>(4, share / row))) : 0;
  // a short call has no rows to fetch ahead
  f.depth = std::min(f.depth, (teams - 1) / (sms * per_sm) + 1);
  f.ring_bytes = f.depth * row;
  f.ctas = std::min(teams, sms * per_sm);
  return f;
}

// ----------------------------------------------------------------- forward

template <typename T, bool WIDE>
__device__ __forceinline__ void load_sum8(const RmsNormArgs& a, long long at, long long c,
                                          int H, float (&v)[kVec]) {
  load8<T, WIDE>(static_cast<const T*>(a.x) + at, c, H, v);
  if (a.residual != nullptr) {
    float r[kVec];
    load8<T, WIDE>(static_cast<const T*>(a.residual) + at, c, H, r);
#pragma unroll
    for (int i = 0; i < kVec; ++i) v[i] += r[i];
  }
}

// A row's normed columns to the outputs the call has.
template <typename T, bool WIDE>
__device__ __forceinline__ void finish8(const RmsNormArgs& a, long long t, long long at,
                                        long long c, int H, float rstd,
                                        const float (&w)[kVec], float (&v)[kVec]) {
#pragma unroll
  for (int i = 0; i < kVec; i += 2) {
    const float2 y = __fmul2_rn(__fmul2_rn(make_float2(v[i], v[i + 1]), make_float2(rstd, rstd)),
                                make_float2(w[i], w[i + 1]));
    v[i] = y.x, v[i + 1] = y.y;
  }
  if (a.out != nullptr) store8<T, WIDE>(static_cast<T*>(a.out) + at, c, H, v);
  if (a.codes != nullptr)
    quantize8<WIDE>(v, c, H, a.codes + at,
                    a.scale + t * static_cast<long long>((a.H + kBlock - 1) / kBlock));
}

// What a thread keeps of a row between its two uses: the sums, or, where nothing is
// added (ADD) to x, x's words.
template <typename T, bool WIDE, bool ADD>
struct Kept {
  float v[kVec];
  __device__ __forceinline__ void load(const RmsNormArgs& a, long long at, long long c, int H) {
    load_sum8<T, WIDE>(a, at, c, H, v);
  }
  __device__ __forceinline__ void get(float (&out)[kVec]) const {
#pragma unroll
    for (int i = 0; i < kVec; ++i) out[i] = v[i];
  }
  __device__ __forceinline__ void keep() {}
};
template <typename T>
struct Kept<T, true, false> {
  uint4 q[sizeof(T) / 2];
  __device__ __forceinline__ void load(const RmsNormArgs& a, long long at, long long c, int H) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i)
      q[i] = c < H ? reinterpret_cast<const uint4*>(static_cast<const T*>(a.x) + at + c)[i]
                   : make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ void get(float (&out)[kVec]) const { word_values<T>(q, out); }
  // The compiler is not to hold the values of one use for the next.
  __device__ __forceinline__ void keep() {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i)
      asm volatile("" : "+r"(q[i].x), "+r"(q[i].y), "+r"(q[i].z), "+r"(q[i].w));
  }
};

// A row in the registers of its team, VPT vectors of eight columns to a thread: inputs
// are read once.  LANES: 32 or 16 lanes of a warp to a row, otherwise (0) a CTA.
template <typename T, bool WIDE, bool ADD, int LANES, int VPT, int THREADS, int CTAS>
__global__ void __launch_bounds__(THREADS, CTAS)
    rms_norm_kernel(const __grid_constant__ RmsNormArgs a) {
  __shared__ float s_sum[32];
  pdl_wait();
  pdl_launch_dependents();
  const int team = LANES > 0 ? LANES : blockDim.x;
  const int member = LANES > 0 ? threadIdx.x % LANES : threadIdx.x;
  const long long t =
      LANES > 0 ? static_cast<long long>(blockIdx.x) * (THREADS / LANES) + threadIdx.x / LANES
                : blockIdx.x;
  if (LANES == 32 && t >= a.T) return;  // whole warps
  // a half warp past the last row goes along with a row of no columns
  const int H = LANES == 16 && t >= a.T ? 0 : a.H;
  const long long at = t * a.H;
  Kept<T, WIDE, ADD> row[VPT];
  float2 ss = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int j = 0; j < VPT; ++j) row[j].load(a, at, (j * team + member) * kVec, H);
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    float v[kVec];
    row[j].get(v);
#pragma unroll
    for (int i = 0; i < kVec; i += 2) {
      const float2 p = make_float2(v[i], v[i + 1]);
      ss = __ffma2_rn(p, p, ss);
    }
  }
  if (ADD && a.sum_out != nullptr) {
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      float v[kVec];
      row[j].get(v);
      store8<T, WIDE>(static_cast<T*>(a.sum_out) + at, (j * team + member) * kVec, H, v);
    }
  }
  const float all = team_sum<LANES>(ss.x + ss.y, s_sum);
  const float rstd = __frsqrt_rn(__fdiv_rn(all, static_cast<float>(a.H)) + a.eps);
  if (a.rstd != nullptr && member == 0 && H > 0) a.rstd[t] = rstd;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int c = (j * team + member) * kVec;
    float v[kVec], w[kVec];
    row[j].keep();
    row[j].get(v);
    load_w8<WIDE>(a.weight, a.w_bf16, c, H, w);
    finish8<T, WIDE>(a, t, at, c, H, rstd, w, v);
  }
}

// Rows too long for registers: read twice.  The sum is stored on the second
// read, so that it may take x's or the residual's place.
template <typename T, bool WIDE>
__global__ void __launch_bounds__(kMaxThreads)
    rms_norm_long_kernel(const __grid_constant__ RmsNormArgs a) {
  __shared__ float s_sum[32];
  pdl_wait();
  pdl_launch_dependents();
  const long long t = blockIdx.x, at = t * a.H;
  // whole warps take part in every step: the codes' maxima go through them
  const long long step = static_cast<long long>(blockDim.x) * kVec;
  const long long first = static_cast<long long>(threadIdx.x) * kVec;
  const long long warp0 = static_cast<long long>(threadIdx.x & ~31u) * kVec;
  float v[kVec], w[kVec], ss = 0.0f;
  for (long long c0 = 0; c0 + warp0 < a.H; c0 += step) {
    load_sum8<T, WIDE>(a, at, c0 + first, a.H, v);
#pragma unroll
    for (int i = 0; i < kVec; ++i) ss = fmaf(v[i], v[i], ss);
  }
  ss = team_sum<0>(ss, s_sum);
  const float rstd = __frsqrt_rn(__fdiv_rn(ss, static_cast<float>(a.H)) + a.eps);
  if (a.rstd != nullptr && threadIdx.x == 0) a.rstd[t] = rstd;
  for (long long c0 = 0; c0 + warp0 < a.H; c0 += step) {
    load_sum8<T, WIDE>(a, at, c0 + first, a.H, v);
    load_w8<WIDE>(a.weight, a.w_bf16, c0 + first, a.H, w);
    if (a.sum_out != nullptr)
      store8<T, WIDE>(static_cast<T*>(a.sum_out) + at, c0 + first, a.H, v);
    finish8<T, WIDE>(a, t, at, c0 + first, a.H, rstd, w, v);
  }
}

template <typename T, bool WIDE, bool ADD, int LANES, int VPT, int THREADS, int CTAS>
cudaError_t launch_rows(const RmsNormArgs& a, int threads, cudaStream_t s) {
  constexpr int kRows = LANES > 0 ? THREADS / LANES : 1;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg =
      pdl_config(dim3((a.T - 1) / kRows + 1), dim3(LANES > 0 ? THREADS : threads), 0, s, attr);
  return cudaLaunchKernelEx(&cfg, rms_norm_kernel<T, WIDE, ADD, LANES, VPT, THREADS, CTAS>, a);
}

// Lanes and vectors per row and, by the registers that are left, CTAs per SM: enough
// bytes on their way, little held behind them.  Without a residual bf16 words take half of
// the values' registers, and rows of many take four vectors a thread, unless there are few
// rows (T=16 H=7168: 2.6 us against 2.2).  us, bf16 T=8192 H=7168, from left to right 2
// vectors and 64 registers, 2 and 40, 4 and 64, 4 and 48: x alone 47.5, 47.6, 38.7, 37.0 (H=1536
// 10.3, 10.4, 10.3, 10.1; its codes 11.6, 11.6, 12.4, 12.3), the codes of a sum 80.9, 67.4, 65.0,
// 63.7, its rows 77.2, 70.0, 70.8, 70.9.  fp32 sums spill at 40 (T=4095 H=2880 31.0, 32.0); x
// alone 17.4, 16.8, 17.4, 17.6, at T=8192 H=7168 81.8, 71.9, 70.7, 71.2.  T=16384 H=1024 bf16 on a
// warp: 64 registers 19.8, 128 23.5 with a residual; T=65536 H=256 on 16 lanes 11.4, on 32
// 12.9, H=128 7.3 and 12.1.
template <typename T, bool WIDE, bool ADD>
cudaError_t launch_in_registers(const RmsNormArgs& a, int vecs, cudaStream_t s) {
  constexpr bool kShort = sizeof(T) == 2;
  if constexpr (WIDE) {
    if (vecs <= 16) return launch_rows<T, WIDE, ADD, 16, 1, 256, kShort ? 8 : 4>(a, 0, s);
    if (vecs <= 32) return launch_rows<T, WIDE, ADD, 16, 2, 256, 4>(a, 0, s);
  }
  if (vecs <= 32) return launch_rows<T, WIDE, ADD, 32, 1, 256, 4>(a, 0, s);
  if (vecs <= 64) return launch_rows<T, WIDE, ADD, 32, 2, 256, ADD ? 4 : 6>(a, 0, s);
  if (vecs <= 128) return launch_rows<T, WIDE, ADD, 32, 4, 256, WIDE && kShort ? 4 : 2>(a, 0, s);
  if constexpr (!ADD) {
    if (vecs > (kShort ? 256 : 512) && a.T > 4 * device_sm_count())
      return launch_rows<T, WIDE, ADD, 0, 4, 256, kShort ? 5 : 4>(
          a, round_up((vecs + 3) / 4, 32), s);
  }
  return launch_rows<T, WIDE, ADD, 0, 2, 512, WIDE && (kShort || !ADD) ? 3 : 2>(
      a, round_up((vecs + 1) / 2, 32), s);
}

template <typename T, bool WIDE>
cudaError_t launch_forward(const RmsNormArgs& a, cudaStream_t s) {
  const int vecs = (a.H - 1) / kVec + 1;
  if (vecs <= 1024) {
    if (a.residual == nullptr && a.sum_out == nullptr)
      return launch_in_registers<T, WIDE, !WIDE>(a, vecs, s);
    return launch_in_registers<T, WIDE, true>(a, vecs, s);
  }
  if (vecs <= 2 * kMaxThreads)
    return launch_rows<T, WIDE, true, 0, 2, kMaxThreads, 1>(a, round_up((vecs + 1) / 2, 32), s);
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = pdl_config(dim3(a.T), dim3(kMaxThreads), 0, s, attr);
  return cudaLaunchKernelEx(&cfg, rms_norm_long_kernel<T, WIDE>, a);
}

// ---------------------------------------------------------------- gradients

// Teams walk the rows a grid apart; a thread keeps its columns' weights and parts of
// dw in registers.  CTA b leaves its part of dw in part[b].
template <typename T, bool WIDE, bool WARP_ROW, int VPT>
__global__ void __launch_bounds__(
    WARP_ROW ? 32 * kWarpRows : kMaxThreads / VPT,
    65536 / grad_regs(sizeof(T), VPT, WIDE) / (WARP_ROW ? 32 * kWarpRows : kMaxThreads / VPT))
    rms_norm_grad_kernel(const __grid_constant__ RmsNormGradArgs a, int depth) {
  __shared__ float s_sum[2][32];
  extern __shared__ uint4 s_ring[];  // and, WARP_ROW, kWarpRows x H floats behind it
  pdl_wait();
  pdl_launch_dependents();
  const int team = WARP_ROW ? 32 : blockDim.x;
  const int member = WARP_ROW ? threadIdx.x & 31 : threadIdx.x;
  const int in_cta = WARP_ROW ? threadIdx.x >> 5 : 0;
  const long long step = WARP_ROW ? static_cast<long long>(gridDim.x) * kWarpRows : gridDim.x;
  long long t = WARP_ROW ? static_cast<long long>(blockIdx.x) * kWarpRows + in_cta : blockIdx.x;
  Ring<T, WIDE, 3, VPT> ring({a.dy, a.h, a.dsum}, s_ring, depth, team, member, a.H, a.T, step);
  ring.clear();
  ring.start(t);
  float2 w[VPT][kVec / 2], dw2[VPT][kVec / 2];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    float f[kVec];
    ring.weights(a.weight, a.w_bf16, j, f);
#pragma unroll
    for (int i = 0; i < kVec / 2; ++i) {
      w[j][i] = make_float2(f[2 * i], f[2 * i + 1]);
      dw2[j][i] = make_float2(0.0f, 0.0f);
    }
  }
  const float inv_h = 1.0f / static_cast<float>(a.H);
  // h is multiplied by rstd before anything else: xhat is of ordinary size whatever h is
  for (int buf = 0; t < a.T; t += step, buf ^= 1) {
    const float rstd = a.rstd[t];
    const float2 rstd2 = make_float2(rstd, rstd);
    float2 dot2 = make_float2(0.0f, 0.0f);
    float2 dy[VPT][kVec / 2], h[VPT][kVec / 2], ds[VPT][kVec / 2];
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
      for (int i = 0; i < kVec / 2; ++i) ds[j][i] = make_float2(0.0f, 0.0f);
    ring.wait();
    // Single elements leave at once and are kept for the second use (T=8192 H=2883, us, read
    // where they are used 116 in bf16 and 92 in fp32: 89 and 88, with the third tensor's
    // among them 93 and 70); words are read from the ring again.
    constexpr bool kSumFirst = !WIDE && sizeof(T) == 4;
    if constexpr (!WIDE) {
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        ring.get(t, 0, j, dy[j]);
        ring.get(t, 1, j, h[j]);
        if (kSumFirst && a.dsum != nullptr) ring.get(t, 2, j, ds[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      if constexpr (WIDE) ring.get(t, 0, j, dy[j]), ring.get(t, 1, j, h[j]);
#pragma unroll
      for (int i = 0; i < kVec / 2; ++i) {
        const float2 xhat = __fmul2_rn(h[j][i], rstd2);
        const float2 p = __fmul2_rn(dy[j][i], xhat);
        dw2[j][i] = __fadd2_rn(dw2[j][i], p);
        dot2 = __ffma2_rn(p, w[j][i], dot2);
        if constexpr (!WIDE) h[j][i] = xhat;
      }
    }
    const float mean = team_sum<WARP_ROW ? 32 : 0>(dot2.x + dot2.y, s_sum[buf]) * inv_h;
    // What xhat (kept) or h (read again) is multiplied by.  rstd * mean is at most dx's size:
    // as one of fp32's small numbers it moves dx by |xhat| 2^-150.  (h scaled by rstd once
    // more instead: T=8192 H=4096 bf16 49.3 -> 50.0 us, H=2880 39.0 -> 40.0.)
    const float k = WIDE ? rstd * mean : mean;
    const float2 k2 = make_float2(-k, -k);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      if constexpr (WIDE) {
        ring.get(t, 0, j, dy[j]);
        ring.get(t, 1, j, h[j]);
      }
      if (!kSumFirst && a.dsum != nullptr) ring.get(t, 2, j, ds[j]);
      float d[kVec];
#pragma unroll
      for (int i = 0; i < kVec / 2; ++i) {
        const float2 v =
            __ffma2_rn(__ffma2_rn(h[j][i], k2, __fmul2_rn(dy[j][i], w[j][i])), rstd2, ds[j][i]);
        d[2 * i] = v.x;
        d[2 * i + 1] = v.y;
      }
      ring.put(static_cast<T*>(a.dx) + t * a.H, j, d);
    }
    ring.next(t);
  }
  float dw[VPT][kVec];
#pragma unroll
  for (int j = 0; j < VPT; ++j)
#pragma unroll
    for (int i = 0; i < kVec / 2; ++i) dw[j][2 * i] = dw2[j][i].x, dw[j][2 * i + 1] = dw2[j][i].y;
  if (a.part == nullptr) return;
  float* part = a.part + static_cast<long long>(blockIdx.x) * a.H;
  if constexpr (WARP_ROW) {
    float* s_dw = reinterpret_cast<float*>(
        s_ring + depth * 3 * VPT * static_cast<int>(sizeof(T) / 2 * blockDim.x));
#pragma unroll
    for (int j = 0; j < VPT; ++j)
      ring.put(s_dw + in_cta * a.H, j, dw[j]);
    __syncthreads();
    for (int c = threadIdx.x; c < a.H; c += blockDim.x) {
      float v = 0.0f;
#pragma unroll
      for (int k = 0; k < kWarpRows; ++k) v += s_dw[k * a.H + c];
      part[c] = v;
    }
  } else {
#pragma unroll
    for (int j = 0; j < VPT; ++j) ring.put(part, j, dw[j]);
  }
}

// Rows too long for registers: dx by reading a row twice, ...
template <typename T, bool WIDE>
__global__ void __launch_bounds__(kMaxThreads)
    rms_norm_grad_long_kernel(const __grid_constant__ RmsNormGradArgs a) {
  __shared__ float s_sum[32];
  pdl_wait();
  pdl_launch_dependents();
  const long long t = blockIdx.x, at = t * a.H;
  // whole warps take part in every step
  const long long step = static_cast<long long>(blockDim.x) * kVec;
  const long long first = static_cast<long long>(threadIdx.x) * kVec;
  const long long warp0 = static_cast<long long>(threadIdx.x & ~31u) * kVec;
  const float rstd = a.rstd[t];
  float dy[kVec], h[kVec], w[kVec], dot = 0.0f;
  auto load = [&](long long c) {
    load8<T, WIDE>(static_cast<const T*>(a.dy) + at, c, a.H, dy);
    load8<T, WIDE>(static_cast<const T*>(a.h) + at, c, a.H, h);
    load_w8<WIDE>(a.weight, a.w_bf16, c, a.H, w);
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      dy[i] *= w[i];
      h[i] *= rstd;
    }
  };
  for (long long c0 = 0; c0 + warp0 < a.H; c0 += step) {
    load(c0 + first);
#pragma unroll
    for (int i = 0; i < kVec; ++i) dot = fmaf(dy[i], h[i], dot);
  }
  const float mean = __fdiv_rn(team_sum<0>(dot, s_sum), static_cast<float>(a.H));
  for (long long c0 = 0; c0 + warp0 < a.H; c0 += step) {
    const long long c = c0 + first;
    load(c);
    float d[kVec], ds[kVec];
    if (a.dsum != nullptr) load8<T, WIDE>(static_cast<const T*>(a.dsum) + at, c, a.H, ds);
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      d[i] = rstd * fmaf(-h[i], mean, dy[i]);
      if (a.dsum != nullptr) d[i] += ds[i];
    }
    store8<T, WIDE>(static_cast<T*>(a.dx) + at, c, a.H, d);
  }
}

// ... and dw's parts by strips of columns: CTA (x, y) adds rows y, y + parts, ...
// of 256 columns.
template <typename T>
__global__ void __launch_bounds__(256)
    rms_norm_dw_long_kernel(const __grid_constant__ RmsNormGradArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const long long c = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (c >= a.H) return;
  float v = 0.0f;
  for (long long t = blockIdx.y; t < a.T; t += gridDim.y)
    v = fmaf(static_cast<float>(static_cast<const T*>(a.dy)[t * a.H + c]),
             static_cast<float>(static_cast<const T*>(a.h)[t * a.H + c]) * a.rstd[t], v);
  a.part[blockIdx.y * static_cast<long long>(a.H) + c] = v;
}

// dw[c] = sum over the parts, in a fixed order: a CTA has 32 columns and up to 32 warps;
// thread (x, y) adds parts y, y + warps, ... of column x in four chains, then a warp the
// sums of a column.  608 parts of 4096 columns: 6 us with the parts' stores (8 columns to
// a CTA and 128 threads to a column, more of it at once but four times the CTAs: 7.4).
__global__ void __launch_bounds__(1024)
    add_parts_kernel(const float* __restrict__ part, int parts, int H, float* __restrict__ dw) {
  __shared__ float s[32][33];
  pdl_wait();
  pdl_launch_dependents();
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const long long c = static_cast<long long>(blockIdx.x) * 32;
  float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (c + x < H) {
    for (int p = y; p < parts; p += 4 * warps) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (p + warps * i < parts) v[i] += part[static_cast<long long>(p + warps * i) * H + c + x];
    }
  }
  s[y][x] = (v[0] + v[1]) + (v[2] + v[3]);
  __syncthreads();
  for (int k = y; k < 32 && c + k < H; k += warps) {
    float sum = x < warps ? s[x][k] : 0.0f;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (x == 0) dw[c + k] = sum;
  }
}

// How a gradient call is cut.  A thread's weights and parts of dw fit its registers
// up to 8192 columns.  The CTAs, and so the parts, are at most those of rows of words.
struct GradForm {
  bool warp_row, in_registers;
  int vpt;
  RowForm rows;
};

size_t warp_dw_bytes(int H) { return static_cast<size_t>(kWarpRows) * H * sizeof(float); }

GradForm grad_form(int T, int H, int es, bool wide, int sms) {
  GradForm f;
  const int vecs = (H - 1) / kVec + 1;
  f.warp_row = vecs <= 64;
  f.in_registers = vecs <= kMaxThreads;
  f.vpt = f.warp_row ? (vecs <= 32 ? 1 : 2) : vecs <= 256 ? 1 : 2;
  const int threads =
      f.warp_row ? 32 * kWarpRows : round_up((vecs + f.vpt - 1) / f.vpt, 32);
  if (f.in_registers) {
    f.rows = row_form(T, es, 3, wide, f.warp_row, f.vpt, threads, grad_regs(es, f.vpt, wide),
                      f.warp_row ? warp_dw_bytes(H) : 0, sms);
  } else {
    f.rows = RowForm{kMaxThreads, 0, std::min(T, sms), 0};
  }
  return f;
}

template <typename T, bool WIDE, bool WARP_ROW, int VPT>
cudaError_t launch_grad_rows(const RmsNormGradArgs& a, const GradForm& f, cudaStream_t s) {
  const size_t smem = f.rows.ring_bytes + (WARP_ROW ? warp_dw_bytes(a.H) : 0);
  static std::atomic<unsigned long long> done{0};
  const cudaError_t err =
      allow_smem(rms_norm_grad_kernel<T, WIDE, WARP_ROW, VPT>, kMostSmem, done);
  if (err != cudaSuccess) return err;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg =
      pdl_config(dim3(f.rows.ctas), dim3(f.rows.threads), smem, s, attr);
  return cudaLaunchKernelEx(&cfg, rms_norm_grad_kernel<T, WIDE, WARP_ROW, VPT>, a, f.rows.depth);
}

template <typename T, bool WIDE>
cudaError_t launch_grad(const RmsNormGradArgs& a, const GradForm& f, cudaStream_t s) {
  cudaLaunchAttribute attr[2];
  cudaError_t e;
  if (f.warp_row) {
    e = f.vpt == 1 ? launch_grad_rows<T, WIDE, true, 1>(a, f, s)
                   : launch_grad_rows<T, WIDE, true, 2>(a, f, s);
  } else if (f.in_registers) {
    e = f.vpt == 1 ? launch_grad_rows<T, WIDE, false, 1>(a, f, s)
                   : launch_grad_rows<T, WIDE, false, 2>(a, f, s);
  } else {
    cudaLaunchConfig_t cfg = pdl_config(dim3(a.T), dim3(kMaxThreads), 0, s, attr);
    e = cudaLaunchKernelEx(&cfg, rms_norm_grad_long_kernel<T, WIDE>, a);
    if (e == cudaSuccess && a.part != nullptr) {
      cfg = pdl_config(dim3((a.H - 1) / 256 + 1, f.rows.ctas), dim3(256), 0, s, attr);
      e = cudaLaunchKernelEx(&cfg, rms_norm_dw_long_kernel<T>, a);
    }
  }
  if (e != cudaSuccess || a.part == nullptr) return e;
  return launch_add_parts(a.part, f.rows.ctas, a.H, a.dw, s);
}

bool on(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

}  // namespace

cudaError_t launch_add_parts(const float* part, int parts, int H, float* dw, cudaStream_t s) {
  // a few rows' parts need no large CTAs
  const int warps = std::max(8, std::min(32, (parts + 3) / 4));
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = pdl_config(dim3((H - 1) / 32 + 1), dim3(32 * warps), 0, s, attr);
  return cudaLaunchKernelEx(&cfg, add_parts_kernel, part, parts, H, dw);
}

cudaError_t launch_rms_norm(const RmsNormArgs& a, int dtype, cudaStream_t s) {
  const bool wide = a.H % kVec == 0 && on(a.x, 16) && on(a.residual, 16) && on(a.weight, 16) &&
                    on(a.sum_out, 16) && on(a.out, 16) && on(a.codes, 8);
  if (dtype == MOE_BF16)
    return wide ? launch_forward<__nv_bfloat16, true>(a, s)
                : launch_forward<__nv_bfloat16, false>(a, s);
  return wide ? launch_forward<float, true>(a, s) : launch_forward<float, false>(a, s);
}

long long rms_norm_grad_parts(int T, int H, int sms) {
  if (T <= 0) return 0;
  return std::max(grad_form(T, H, 2, true, sms).rows.ctas,
                  grad_form(T, H, 4, true, sms).rows.ctas);
}

cudaError_t launch_rms_norm_grad(const RmsNormGradArgs& a, int dtype, int sms, cudaStream_t s) {
  const bool wide = a.H % kVec == 0 && on(a.dy, 16) && on(a.h, 16) && on(a.weight, 16) &&
                    on(a.dsum, 16) && on(a.dx, 16) && on(a.part, 16);
  const GradForm f = grad_form(a.T, a.H, dtype == MOE_BF16 ? 2 : 4, wide, sms);
  if (dtype == MOE_BF16)
    return wide ? launch_grad<__nv_bfloat16, true>(a, f, s)
                : launch_grad<__nv_bfloat16, false>(a, f, s);
  return wide ? launch_grad<float, true>(a, f, s) : launch_grad<float, false>(a, f, s);
}

}  // namespace moe
