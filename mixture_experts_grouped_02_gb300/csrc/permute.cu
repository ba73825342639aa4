// permute.cu -- token rows to the expert-sorted list and back, with their
// gradients.
//
// With i = t*K + k the flat index of token t's k-th choice, slot(i) =
// inv_perm[i] its place in the padded list moe_align makes and sorted_ids its
// inverse:
//   permute             xs[slot(i)] = x[i / K], rows of padding slots zero
//   its gradient        dx[t] = sum_k dxs[slot(tK + k)]
//   unpermute           out[t] = sum_k w[t, k] * y[slot(tK + k)]
//   its gradients       dy[slot(i)] = w[i] * dout[i / K], padding rows zero
//                       dw[i] = dout[i / K] . y[slot(i)]
// Sums run in fp32 in k order (dw: lane partial sums and a fixed tree) and are
// rounded once to the rows' type, so results do not depend on the schedule.
// An assignment to another shard's expert (slot < 0) adds nothing and gets
// dw = 0.  Sources: the "Current PyTorch path" of "factor_moe_fused_gemm.cu"
// (gather of the routed rows, index_add of the weighted ones), whose autograd
// these gradients are.
//
// All four move bytes and compute next to nothing: HBM bounds them, and the
// launch bounds the smallest.
#include <cuda_bf16.h>

#include <algorithm>

#include "bounds.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
// Slots a CTA looks at for padding rows: padding comes in runs (an expert's
// last block, the tail of the list), so a short list takes one slot per CTA
// (the 120 padding rows of one token's list took 14 us as eight rows a warp,
// 2 us so), and a long one up to a warp's worth, which keeps the CTAs few.
int pad_slots(long long cap) {
  return static_cast<int>(std::max(1ll, std::min(32ll, cap / (device_sm_count() * 16))));
}

// A run of V elements of type T, loaded and stored as one word.
template <int BYTES>
struct Word;
template <>
struct Word<16> {
  using type = uint4;
};
template <>
struct Word<4> {
  using type = uint32_t;
};
template <>
struct Word<2> {
  using type = uint16_t;
};
template <>
struct Word<1> {
  using type = uint8_t;
};

template <typename T, int V>
__device__ __forceinline__ void unpack(const typename Word<sizeof(T) * V>::type& w, float (&f)[V]) {
  if constexpr (V == 1) {
    f[0] = static_cast<float>(*reinterpret_cast<const T*>(&w));
  } else if constexpr (sizeof(T) == 2) {
    const uint32_t p[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(p[i] << 16);
      f[2 * i + 1] = __uint_as_float(p[i] & 0xffff0000u);
    }
  } else {
    f[0] = __uint_as_float(w.x);
    f[1] = __uint_as_float(w.y);
    f[2] = __uint_as_float(w.z);
    f[3] = __uint_as_float(w.w);
  }
}

// One rounding to nearest even from fp32 to the rows' type.
template <typename T, int V>
__device__ __forceinline__ typename Word<sizeof(T) * V>::type pack(const float (&f)[V]) {
  if constexpr (V == 1) {
    const T v = static_cast<T>(f[0]);
    return *reinterpret_cast<const typename Word<sizeof(T)>::type*>(&v);
  } else if constexpr (sizeof(T) == 2) {
    uint32_t p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      p[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(p[0], p[1], p[2], p[3]);
  } else {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
}

// Zero rows of the padding slots among slots [job * per, job * per + per),
// per <= 32, by one CTA.
template <typename W>
__device__ __forceinline__ void zero_padding(const int32_t* __restrict__ sorted_ids, long long job,
                                             int per, long long cap, int n_assign, int row_words,
                                             W* __restrict__ rows) {
  const int lane = threadIdx.x & 31;
  const long long s0 = job * per;
  const bool pad = lane < per && s0 + lane < cap && sorted_ids[s0 + lane] >= n_assign;
  unsigned todo = __ballot_sync(0xffffffffu, pad);
  while (todo != 0) {
    const int u = __ffs(todo) - 1;
    todo &= todo - 1;
    W* row = rows + (s0 + u) * row_words;
    for (int c = threadIdx.x; c < row_words; c += kThreads) row[c] = W{};
  }
}

// Jobs [0, T * chunks): U * 256 words of a token's row, read once and written
// to the slots of its K choices.  Jobs after them: padding rows.
template <typename W, int U>
__global__ void __launch_bounds__(kThreads)
    permute_kernel(const W* __restrict__ x, int T, int K, int row_words, int chunks, int pad_per,
                   const int32_t* __restrict__ inv_perm, const int32_t* __restrict__ sorted_ids,
                   long long cap, W* __restrict__ xs, const int32_t* status) {
  pdl_wait();
  pdl_launch_dependents();
  if (status != nullptr && *status != 0) return;
  const long long token_jobs = static_cast<long long>(T) * chunks;
  if (blockIdx.x >= token_jobs) {
    zero_padding(sorted_ids, blockIdx.x - token_jobs, pad_per, cap, T * K, row_words, xs);
    return;
  }
  const int t = static_cast<int>(blockIdx.x / static_cast<unsigned>(chunks));
  const int c = static_cast<int>(blockIdx.x - static_cast<unsigned>(t) * chunks) * (U * kThreads) +
                threadIdx.x;
  W v[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (c + u * kThreads < row_words)
      v[u] = x[static_cast<long long>(t) * row_words + c + u * kThreads];
  for (int k = 0; k < K; ++k) {
    const long long slot = inv_perm[static_cast<long long>(t) * K + k];
    if (slot < 0 || !in_bounds(slot < cap, status)) continue;
    W* row = xs + slot * row_words + c;
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (c + u * kThreads < row_words) row[u * kThreads] = v[u];
  }
}

// out[t] = sum_k w[t, k] * y[slot(tK + k)] (w null: all one).  Words of the
// output are dealt to threads across token boundaries, U words 256 apart to a
// thread, and U * KB loads are in flight before the first is added; `group`
// tokens make up one grid row, which keeps the word index in 32 bits.
template <typename T, int V, int U, int KB>
__global__ void __launch_bounds__(kThreads)
    unpermute_kernel(const T* __restrict__ y_, const float* __restrict__ weights, int tokens,
                     int K, int row_words, int group, const int32_t* __restrict__ inv_perm,
                     long long cap, T* __restrict__ out_, const int32_t* status) {
  using W = typename Word<sizeof(T) * V>::type;
  pdl_wait();
  pdl_launch_dependents();
  if (status != nullptr && *status != 0) return;
  const W* y = reinterpret_cast<const W*>(y_);
  W* out = reinterpret_cast<W*>(out_);
  const unsigned idx = blockIdx.x * (U * kThreads) + threadIdx.x;
  for (long long g = blockIdx.y; g * group < tokens; g += gridDim.y) {
    float acc[U][V];
    long long t[U];
    int c[U];
    bool ok[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const unsigned i = idx + u * kThreads;
      const unsigned tl = i / static_cast<unsigned>(row_words);
      c[u] = static_cast<int>(i - tl * row_words);
      t[u] = g * group + tl;
      ok[u] = tl < static_cast<unsigned>(group) && t[u] < tokens;
#pragma unroll
      for (int j = 0; j < V; ++j) acc[u][j] = 0.0f;
    }
    for (int k0 = 0; k0 < K; k0 += KB) {
      W v[U][KB];
      bool held[U][KB];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < KB; ++j) {
          held[u][j] = false;
          if (ok[u] && k0 + j < K) {
            const long long slot = inv_perm[t[u] * K + k0 + j];
            held[u][j] = slot >= 0 && in_bounds(slot < cap, status);
            if (held[u][j]) v[u][j] = y[slot * row_words + c[u]];
          }
        }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < KB; ++j)
          if (held[u][j]) {
            const float w = weights != nullptr ? weights[t[u] * K + k0 + j] : 1.0f;
            float f[V];
            unpack<T, V>(v[u][j], f);
#pragma unroll
            for (int i = 0; i < V; ++i) acc[u][i] = fmaf(w, f[i], acc[u][i]);
          }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (ok[u]) out[t[u] * row_words + c[u]] = pack<T, V>(acc[u]);
  }
}

// The same for rows that do not move in 16-byte words: U * 256 elements of one
// token to a CTA, so that slots and weights are looked up once per choice and
// not per element (H = 1999, K = 2, T = 4096 in bf16: 48 -> 15 us).
template <typename T, int U>
__global__ void __launch_bounds__(kThreads)
    unpermute_elems_kernel(const T* __restrict__ y, const float* __restrict__ weights, int K,
                           int H, int chunks, const int32_t* __restrict__ inv_perm,
                           long long cap, T* __restrict__ out, const int32_t* status) {
  pdl_wait();
  pdl_launch_dependents();
  if (status != nullptr && *status != 0) return;
  const int t = static_cast<int>(blockIdx.x / static_cast<unsigned>(chunks));
  const int c = static_cast<int>(blockIdx.x - static_cast<unsigned>(t) * chunks) * (U * kThreads) +
                threadIdx.x;
  float acc[U];
#pragma unroll
  for (int u = 0; u < U; ++u) acc[u] = 0.0f;
  for (int k = 0; k < K; ++k) {
    const long long i = static_cast<long long>(t) * K + k;
    const long long slot = inv_perm[i];
    if (slot < 0 || !in_bounds(slot < cap, status)) continue;
    const float w = weights != nullptr ? weights[i] : 1.0f;
    const T* row = y + slot * H + c;
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (c + u * kThreads < H)
        acc[u] = fmaf(w, static_cast<float>(row[u * kThreads]), acc[u]);
  }
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (c + u * kThreads < H)
      out[static_cast<long long>(t) * H + c + u * kThreads] = static_cast<T>(acc[u]);
}

// A warp per assignment, its dy row and its dw; the CTAs from `pad0` on take
// padding rows.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads)
    unpermute_backward_kernel(const T* __restrict__ dout_, const T* __restrict__ y_,
                              const float* __restrict__ weights, int n_assign, int K,
                              int row_words, unsigned pad0, int pad_per,
                              const int32_t* __restrict__ inv_perm,
                              const int32_t* __restrict__ sorted_ids, long long cap,
                              T* __restrict__ dy_, float* __restrict__ dw,
                              const int32_t* status) {
  using W = typename Word<sizeof(T) * V>::type;
  constexpr int U = 4;  // words of a lane in flight
  pdl_wait();
  pdl_launch_dependents();
  if (status != nullptr && *status != 0) return;
  W* dy = reinterpret_cast<W*>(dy_);
  if (blockIdx.x >= pad0) {
    zero_padding(sorted_ids, blockIdx.x - pad0, pad_per, cap, n_assign, row_words, dy);
    return;
  }
  const int lane = threadIdx.x & 31;
  const int job = static_cast<int>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (job >= n_assign) return;
  const long long slot = inv_perm[job];
  if (slot < 0 || !in_bounds(slot < cap, status)) {
    if (lane == 0) dw[job] = 0.0f;
    return;
  }
  const float w = weights[job];
  const W* g = reinterpret_cast<const W*>(dout_) + static_cast<long long>(job / K) * row_words;
  const W* y = reinterpret_cast<const W*>(y_) + slot * row_words;
  dy += slot * row_words;
  // four chains to a lane, of H / 128 terms each: the error grows with a chain's
  // length (T=4095 H=4096 K=2 fp32: 1.2e-7 relative, 2.1e-7 with one chain of
  // H / 32; the time is the same, 88 us)
  float dots[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int c0 = lane; c0 < row_words; c0 += 32 * U) {
    W gv[U], yv[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (c0 + 32 * u < row_words) {
        gv[u] = g[c0 + 32 * u];
        yv[u] = y[c0 + 32 * u];
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (c0 + 32 * u < row_words) {
        float gf[V], yf[V];
        unpack<T, V>(gv[u], gf);
        unpack<T, V>(yv[u], yf);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          float& dot = dots[V == 1 ? u : i & 3];
          dot = fmaf(gf[i], yf[i], dot);
          gf[i] *= w;
        }
        dy[c0 + 32 * u] = pack<T, V>(gf);
      }
  }
  float dot = (dots[0] + dots[1]) + (dots[2] + dots[3]);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
  if (lane == 0) dw[job] = dot;
}

// Largest power of two up to 16 that divides the row and every address.
int word_bytes(long long row_bytes, const void* a, const void* b, const void* c = nullptr) {
  const uintptr_t all = static_cast<uintptr_t>(row_bytes) | reinterpret_cast<uintptr_t>(a) |
                        reinterpret_cast<uintptr_t>(b) | reinterpret_cast<uintptr_t>(c) | 16u;
  return static_cast<int>(all & (~all + 1));
}

long long pad_jobs(long long cap, int per) { return (cap + per - 1) / per; }

template <typename W>
cudaError_t permute_as(const void* x, int T, int K, long long row_bytes, const int32_t* inv_perm,
                       const int32_t* sorted_ids, long long cap, void* xs, const int32_t* status,
                       cudaStream_t s) {
  const int row_words = static_cast<int>(row_bytes / sizeof(W));
  constexpr int U = sizeof(W) == 16 ? 1 : 8;
  const int chunks = (row_words + U * kThreads - 1) / (U * kThreads);
  const int per = pad_slots(cap);
  const long long grid = static_cast<long long>(T) * chunks + pad_jobs(cap, per);
  if (grid > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = pdl_config(dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, s, attr);
  return cudaLaunchKernelEx(&cfg, permute_kernel<W, U>, static_cast<const W*>(x), T, K, row_words,
                            chunks, per, inv_perm, sorted_ids, cap, static_cast<W*>(xs), status);
}

template <typename T, int V, int U, int KB>
cudaError_t unpermute_as(const void* y, const float* weights, int tokens, int K, int H,
                         const int32_t* inv_perm, long long cap, void* out, const int32_t* status,
                         cudaStream_t s) {
  const int row_words = H / V;
  const int group = std::min(tokens, std::max(1, (1 << 20) / row_words));
  const long long rows = (static_cast<long long>(tokens) + group - 1) / group;
  const long long per = U * kThreads;
  const dim3 grid(static_cast<unsigned>((group * static_cast<long long>(row_words) + per - 1) / per),
                  static_cast<unsigned>(std::min(rows, 65535ll)));
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = pdl_config(grid, dim3(kThreads), 0, s, attr);
  return cudaLaunchKernelEx(&cfg, unpermute_kernel<T, V, U, KB>, static_cast<const T*>(y),
                            weights, tokens, K, row_words, group, inv_perm, cap,
                            static_cast<T*>(out), status);
}

template <typename T>
cudaError_t unpermute_elems(const void* y, const float* weights, int tokens, int K, int H,
                            const int32_t* inv_perm, long long cap, void* out,
                            const int32_t* status, cudaStream_t s) {
  constexpr int U = 8;
  const int chunks = static_cast<int>((H + static_cast<long long>(U) * kThreads - 1) /
                                      (U * kThreads));
  const long long grid = static_cast<long long>(tokens) * chunks;
  if (grid > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg =
      pdl_config(dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, s, attr);
  return cudaLaunchKernelEx(&cfg, unpermute_elems_kernel<T, U>, static_cast<const T*>(y), weights,
                            K, H, chunks, inv_perm, cap, static_cast<T*>(out), status);
}

// 16-byte words: the loads of a token's choices in flight together, eight at
// a time, and of two words of the output where the choices are few.
template <typename T, int V>
cudaError_t unpermute_by_k(const void* y, const float* w, int tokens, int K, int H,
                           const int32_t* inv_perm, long long cap, void* out,
                           const int32_t* status, cudaStream_t s) {
  if (K <= 2) return unpermute_as<T, V, 2, 2>(y, w, tokens, K, H, inv_perm, cap, out, status, s);
  if (K <= 4) return unpermute_as<T, V, 1, 4>(y, w, tokens, K, H, inv_perm, cap, out, status, s);
  return unpermute_as<T, V, 1, 8>(y, w, tokens, K, H, inv_perm, cap, out, status, s);
}

template <typename T, int V>
cudaError_t unpermute_backward_as(const void* dout, const void* y, const float* weights,
                                  int tokens, int K, int H, const int32_t* inv_perm,
                                  const int32_t* sorted_ids, long long cap, void* dy, float* dw,
                                  const int32_t* status, cudaStream_t s) {
  const unsigned pad0 = static_cast<unsigned>((tokens * K + kWarps - 1) / kWarps);
  const int per = pad_slots(cap);
  const unsigned grid = pad0 + static_cast<unsigned>(pad_jobs(cap, per));
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = pdl_config(dim3(grid), dim3(kThreads), 0, s, attr);
  return cudaLaunchKernelEx(&cfg, unpermute_backward_kernel<T, V>, static_cast<const T*>(dout),
                            static_cast<const T*>(y), weights, tokens * K, K, H / V, pad0,
                            per, inv_perm, sorted_ids, cap, static_cast<T*>(dy), dw, status);
}

}  // namespace

cudaError_t launch_permute(const void* x, int T, long long row_bytes, int K,
                           const int32_t* inv_perm, const int32_t* sorted_ids, long long cap,
                           void* xs, const int32_t* status, cudaStream_t s) {
  switch (word_bytes(row_bytes, x, xs)) {
    case 16:
      return permute_as<uint4>(x, T, K, row_bytes, inv_perm, sorted_ids, cap, xs, status, s);
    case 8:
    case 4:
      return permute_as<uint32_t>(x, T, K, row_bytes, inv_perm, sorted_ids, cap, xs, status, s);
    case 2:
      return permute_as<uint16_t>(x, T, K, row_bytes, inv_perm, sorted_ids, cap, xs, status, s);
    default:
      return permute_as<uint8_t>(x, T, K, row_bytes, inv_perm, sorted_ids, cap, xs, status, s);
  }
}

cudaError_t launch_unpermute(const void* y, int dtype, const float* weights, int T, int K, int H,
                             const int32_t* inv_perm, long long cap, void* out,
                             const int32_t* status, cudaStream_t s) {
  const bool bf16 = dtype == MOE_BF16;
  const bool wide = word_bytes(static_cast<long long>(H) * (bf16 ? 2 : 4), y, out) == 16;
  if (bf16)
    return wide ? unpermute_by_k<__nv_bfloat16, 8>(y, weights, T, K, H, inv_perm, cap, out, status, s)
                : unpermute_elems<__nv_bfloat16>(y, weights, T, K, H, inv_perm, cap, out, status, s);
  return wide ? unpermute_by_k<float, 4>(y, weights, T, K, H, inv_perm, cap, out, status, s)
              : unpermute_elems<float>(y, weights, T, K, H, inv_perm, cap, out, status, s);
}

cudaError_t launch_unpermute_backward(const void* dout, const void* y, int dtype,
                                      const float* weights, int T, int K, int H,
                                      const int32_t* inv_perm, const int32_t* sorted_ids,
                                      long long cap, void* dy, float* dw, const int32_t* status,
                                      cudaStream_t s) {
  const bool bf16 = dtype == MOE_BF16;
  const bool wide = word_bytes(static_cast<long long>(H) * (bf16 ? 2 : 4), dout, y, dy) == 16;
  if (bf16)
    return wide ? unpermute_backward_as<__nv_bfloat16, 8>(dout, y, weights, T, K, H, inv_perm,
                                                          sorted_ids, cap, dy, dw, status, s)
                : unpermute_backward_as<__nv_bfloat16, 1>(dout, y, weights, T, K, H, inv_perm,
                                                          sorted_ids, cap, dy, dw, status, s);
  return wide ? unpermute_backward_as<float, 4>(dout, y, weights, T, K, H, inv_perm, sorted_ids,
                                                cap, dy, dw, status, s)
              : unpermute_backward_as<float, 1>(dout, y, weights, T, K, H, inv_perm, sorted_ids,
                                                cap, dy, dw, status, s);
}

}  // namespace moe
