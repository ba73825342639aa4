// gemm_fp8b.cu -- products of e4m3 operands with fp32 block scales, plain or
// one per expert of a sorted list, on tcgen05:
//
//   out[m, n] = sum_b sa[m, b] * sb[n / 128, b] * sum_{k in block b} a[m, k] * w[n, k]
//
// with b running over the blocks of 128 elements along K.  The scales are
// fp32 and change with b, so a block's products cannot stay in one
// accumulator: the tensor core sums a block (K = 128, four MMAs) into a TMEM
// buffer of its own, and the epilogue warps multiply it by sa * sb and add it
// to fp32 registers while the tensor core fills the other buffer.  A row's
// scale is one register of the thread that owns the row, and a 128-column
// half of the tile has one weight scale, so this costs one packed
// fma.rn.f32x2 for two elements.
//
// Layout per CTA (one per SM, persistent, tiles walked in bands as in
// sched.cuh):
//  * tile = 128 rows of a x 256 weight rows; the columns past N in the last
//    tile are left out of the MMA's N;
//  * four stages of one scale block each: A 128 x 128 bytes (16 KB; 32 rows
//    when the block has at most 32 valid rows), B 256 x 128 bytes (32 KB),
//    128-byte swizzled, by TMA.  K past the tensor reads as zero codes;
//  * TMEM: two 256-column fp32 buffers;
//  * warp 0 TMA, warp 1 MMA, warps 2-9 epilogue: warp w reads the lane
//    quarter w % 4 and one half of the columns, 128 fp32 sums per thread.
//    A warp whose 32 rows are all padding only keeps the barriers.
//
// Every mbarrier wait is bounded, as in the other GEMMs: a thread that gives
// up raises the CTA's abort flag and the kernel records MOE_ERR_TIMEOUT,
// drains and frees its TMEM.
#include <cuda_bf16.h>

#include "bounds.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "sched.cuh"

namespace moe {
namespace {

struct Cfg {
  static constexpr int kBM = 128;
  static constexpr int kBN = 256;
  static constexpr int kBK = 128;
  static constexpr int kUmmaK = 32;
  static constexpr int kStages = 4;
  static constexpr int kABytes = kBM * kBK;
  static constexpr int kAShortRows = 32;
  static constexpr int kAShortBytes = kAShortRows * kBK;
  static constexpr int kBBytes = kBN * kBK;
  static constexpr int kTmemCols = 2 * kBN;
  static constexpr int kMmaWarp = 1;
  static constexpr int kEpiWarps = 8;
  static constexpr int kThreads = (2 + kEpiWarps) * 32;
  static constexpr int kSmemBytes = kStages * (kABytes + kBBytes) + 1024;
};

// Row block `mb` of the call: expert, first row, valid rows.
struct RowBlock {
  int e, r0, valid;
};

__device__ __forceinline__ RowBlock row_block(const Fp8bArgs& a, int mb) {
  RowBlock r;
  if (a.block_info == nullptr) {
    r.e = 0;
    r.r0 = mb * Cfg::kBM;
    r.valid = min(Cfg::kBM, a.M - r.r0);
    return r;
  }
  // align blocks of up to 256 rows are read as `subs` row blocks
  const int b = mb / a.subs;
  const int4 bi = reinterpret_cast<const int4*>(a.block_info)[b];
  const int off = (mb - b * a.subs) * Cfg::kBM;
  r.e = bi.x;
  r.r0 = bi.z + off;
  r.valid = block_in_bounds(bi, a.E, a.cap, a.subs * Cfg::kBM, a.status)
                ? max(0, min(Cfg::kBM, bi.w - off))
                : 0;
  return r;
}

__device__ __forceinline__ uint64_t pack2(uint32_t lo, uint32_t hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(lo), "r"(hi));
  return v;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
  uint32_t a, b;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(v));
  lo = __uint_as_float(a);
  hi = __uint_as_float(b);
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// 128 sums of a row to columns [col, col + 128) of out, those below N.
__device__ __forceinline__ void store_row(const Fp8bArgs& a, long long row, int col,
                                          const uint64_t (&acc)[64]) {
  const int n = min(128, a.N - col);
  if (a.out_bf16) {
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.out) + row * a.N + col;
    if (a.wide_out) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if (8 * i < n) {
          uint32_t p[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float lo, hi;
            unpack2(acc[4 * i + j], lo, hi);
            const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
            p[j] = *reinterpret_cast<const uint32_t*>(&h);
          }
          reinterpret_cast<uint4*>(o)[i] = make_uint4(p[0], p[1], p[2], p[3]);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 64; ++i) {
        float lo, hi;
        unpack2(acc[i], lo, hi);
        if (2 * i < n) o[2 * i] = __float2bfloat16_rn(lo);
        if (2 * i + 1 < n) o[2 * i + 1] = __float2bfloat16_rn(hi);
      }
    }
    return;
  }
  float* o = static_cast<float*>(a.out) + row * a.N + col;
  if (a.wide_out) {
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      if (4 * i < n) {
        float4 v;
        unpack2(acc[2 * i], v.x, v.y);
        unpack2(acc[2 * i + 1], v.z, v.w);
        reinterpret_cast<float4*>(o)[i] = v;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 64; ++i) {
      float lo, hi;
      unpack2(acc[i], lo, hi);
      if (2 * i < n) o[2 * i] = lo;
      if (2 * i + 1 < n) o[2 * i + 1] = hi;
    }
  }
}

__global__ void __launch_bounds__(Cfg::kThreads, 1)
    fp8b_gemm_kernel(const __grid_constant__ Fp8bArgs a, const __grid_constant__ CUtensorMap tmA,
                     const __grid_constant__ CUtensorMap tmAShort,
                     const __grid_constant__ CUtensorMap tmB) {
  using C = Cfg;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full_bar[C::kStages];
  __shared__ __align__(8) uint64_t empty_bar[C::kStages];
  __shared__ __align__(8) uint64_t accf_bar[2];
  __shared__ __align__(8) uint64_t acce_bar[2];
  __shared__ __align__(8) uint64_t drain_bar;
  __shared__ uint32_t s_tmem_base;
  __shared__ int s_skip;
  __shared__ volatile int s_abort;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t smemA = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t smemB = smemA + C::kStages * C::kABytes;

  pdl_wait();
  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    s_skip = (a.status != nullptr && *reinterpret_cast<volatile int32_t*>(a.status) != 0);
    s_abort = 0;
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(smem_u32(&full_bar[i]), 1);
      mbar_init(smem_u32(&empty_bar[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&accf_bar[i]), 1);
      mbar_init(smem_u32(&acce_bar[i]), C::kEpiWarps);
    }
    mbar_init(smem_u32(&drain_bar), 1);
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  __syncthreads();
  if (s_skip) return;
  if (warp == C::kMmaWarp) tmem_alloc(smem_u32(&s_tmem_base), C::kTmemCols);
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmAShort);
    tma_prefetch_desc(&tmB);
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = s_tmem_base;

  const int num_blocks =
      a.block_info == nullptr
          ? a.max_blocks
          : checked_num_blocks(*a.num_blocks, a.max_blocks, a.status) * a.subs;
  const int total = num_blocks * a.n_tiles;
  const uint64_t to = a.timeout_ns;

  if (warp == 0) {
    // ------------------------------------------------------- TMA producer
    if (lane == 0 && !a.starve) {
      uint32_t stage = 0, phase = 0;
      long long issued = 0;
      bool ok = true;
      for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
        const Tile t = decode_tile(tile, num_blocks, a);
        const RowBlock r = row_block(a, t.mb);
        if (r.valid <= 0) continue;
        const bool short_a = r.valid <= C::kAShortRows;
        const uint32_t tx = C::kBBytes + (short_a ? C::kAShortBytes : C::kABytes);
        const int w_row = r.e * a.N + t.nt * C::kBN;
        for (int kt = 0; kt < a.k_tiles; ++kt) {
          if (!mbar_wait_bounded(smem_u32(&empty_bar[stage]), phase ^ 1, &s_abort, to)) {
            ok = false;
            break;
          }
          const uint32_t fb = smem_u32(&full_bar[stage]);
          mbar_arrive_expect_tx(fb, tx);
          tma_load_2d(smemA + stage * C::kABytes, short_a ? &tmAShort : &tmA, fb, kt * C::kBK,
                      r.r0);
          tma_load_2d(smemB + stage * C::kBBytes, &tmB, fb, kt * C::kBK, w_row);
          ++issued;
          if (++stage == C::kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      if (!ok) {
        const long long first = issued > C::kStages ? issued - C::kStages : 0;
        for (long long n = first; n < issued; ++n)
          drain_wait(smem_u32(&full_bar[n % C::kStages]),
                     static_cast<uint32_t>((n / C::kStages) & 1), to / 4);
      }
    }
    __syncwarp();
  } else if (warp == C::kMmaWarp) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      uint32_t stage = 0, phase = 0, buf = 0, buf_phase = 0;
      bool ok = true;
      for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
        const Tile t = decode_tile(tile, num_blocks, a);
        if (row_block(a, t.mb).valid <= 0) continue;
        const int n = min(C::kBN, (a.N - t.nt * C::kBN + 15) & ~15);
        const uint32_t idesc = make_idesc(0, C::kBM, n);  // e4m3 x e4m3
        for (int kt = 0; kt < a.k_tiles; ++kt) {
          if (!mbar_wait_bounded(smem_u32(&acce_bar[buf]), buf_phase ^ 1, &s_abort, to) ||
              !mbar_wait_bounded(smem_u32(&full_bar[stage]), phase, &s_abort, to)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint32_t a_base = smemA + stage * C::kABytes;
          const uint32_t b_base = smemB + stage * C::kBBytes;
          const uint32_t d_tmem = tmem_base + buf * C::kBN;
#pragma unroll
          for (int k = 0; k < C::kBK / C::kUmmaK; ++k)
            umma_f8(d_tmem, sw128_kmajor_desc(a_base + k * C::kUmmaK),
                    sw128_kmajor_desc(b_base + k * C::kUmmaK), idesc, k > 0 ? 1u : 0u);
          umma_commit(smem_u32(&empty_bar[stage]));
          umma_commit(smem_u32(&accf_bar[buf]));
          if (++stage == C::kStages) {
            stage = 0;
            phase ^= 1;
          }
          buf ^= 1;
          if (buf == 0) buf_phase ^= 1;
        }
      }
      if (!ok) {
        umma_commit(smem_u32(&drain_bar));
        drain_wait(smem_u32(&drain_bar), 0, to / 4);
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;
    const int half = (warp - 2) >> 2;
    uint32_t buf = 0, buf_phase = 0;
    bool ok = true;
    for (int tile = blockIdx.x; tile < total && ok; tile += gridDim.x) {
      const Tile t = decode_tile(tile, num_blocks, a);
      const RowBlock r = row_block(a, t.mb);
      if (r.valid <= 0) continue;
      const int local = q * 32 + lane;
      const long long row = r.r0 + local;
      const bool row_ok = local < r.valid;
      const int col = t.nt * C::kBN + half * 128;
      // warps without a row or a column of the output only keep the barriers
      const bool live = q * 32 < r.valid && col < a.N;
      const float* sa = a.a_scale + (row_ok ? row : r.r0) * a.k_tiles;
      const float* sb = a.w_scale +
                        (static_cast<long long>(r.e) * a.n_scales +
                         min(col, a.N - 1) / 128) * a.k_tiles;
      uint64_t acc[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i] = 0;
      float s_next = live ? __ldg(sa) * __ldg(sb) : 0.0f;
      for (int kt = 0; kt < a.k_tiles; ++kt) {
        const uint32_t s_bits = __float_as_uint(s_next);
        if (live && kt + 1 < a.k_tiles) s_next = __ldg(sa + kt + 1) * __ldg(sb + kt + 1);
        const int good = mbar_wait_bounded(smem_u32(&accf_bar[buf]), buf_phase, &s_abort, to);
        if (!__all_sync(0xffffffffu, good)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        if (live) {
          const uint64_t s2 = pack2(s_bits, s_bits);
          const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                                 buf * C::kBN + half * 128;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t v[32];
            tmem_ld32(taddr + 32 * c, v);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i)
              acc[16 * c + i] = fma2(pack2(v[2 * i], v[2 * i + 1]), s2, acc[16 * c + i]);
          }
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&acce_bar[buf]));
        buf ^= 1;
        if (buf == 0) buf_phase ^= 1;
      }
      if (ok && live && row_ok) store_row(a, row, col, acc);
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if (threadIdx.x == 0 && s_abort) report_error(a.status, MOE_ERR_TIMEOUT);
  if (warp == C::kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem_base, C::kTmemCols);
  }
}

}  // namespace

cudaError_t launch_fp8b_gemm(Fp8bArgs a, const CUtensorMap& tmA, const CUtensorMap& tmAShort,
                             const CUtensorMap& tmB, int sms, cudaStream_t s) {
  using C = Cfg;
  a.n_tiles = (a.N + C::kBN - 1) / C::kBN;
  a.band = a.n_tiles < 8 ? a.n_tiles : 8;
  const long long tiles = static_cast<long long>(a.max_blocks) * a.subs * a.n_tiles;
  if (tiles > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  cudaError_t err = cudaFuncSetAttribute(
      fp8b_gemm_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
  if (err != cudaSuccess) return err;
  const int grid = static_cast<int>(tiles < sms ? tiles : sms);
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = pdl_config(dim3(grid), dim3(C::kThreads), C::kSmemBytes, s, attr);
  return cudaLaunchKernelEx(&cfg, fp8b_gemm_kernel, a, tmA, tmAShort, tmB);
}

}  // namespace moe
