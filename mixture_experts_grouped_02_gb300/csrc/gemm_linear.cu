// gemm_linear.cu -- products of bf16 operands with what follows them in the
// kernel (linear_epi.cuh):
//
//   out = epilogue of sum over k of A(m, k) B(n, k)
//
// on tcgen05 with fp32 accumulators in TMEM.  A linear layer's three products are
// one kernel with operands that lie differently in memory: y = x w^T has both by
// rows, dx = dz w has w's reduction along its rows, dw = dz^T x both operands';
// tcgen05 reads such a tile as it lies (M/N-major), so nothing is transposed.
//
// Two kernels:
//  * linear_kernel: one CTA per tile of 128 rows x BN weight rows, 64 or 128, or
//    (64) a cluster of 2 to 8 CTAs that share a tile's K range and add the
//    partial sums through distributed shared memory, in rank order, for products
//    with fewer tiles than SMs;
//  * linear_pair_kernel: a CTA pair (cta_group::2) per tile of 256 x 256, 224 or 128,
//    each CTA with half of the weight rows: what a CTA's shared memory takes in (some
//    78 bytes a clock, measured) bounds the smaller tiles, 32 KB per K step for 128 x
//    128 outputs in one CTA, 24 KB on a pair of 256 x 128, and for 256 x 256 the MMAs'
//    512 clocks bound a K step.  Measured K steps, us: 0.16 for 128 x 64 in a CTA, 0.22 for
//    128 x 128, 0.18 for a pair's 256 x 128 and 0.285 for its 256 x 256, which is 98 % of
//    the bf16 rate (8192 x 4096 x 4096 143 us, 141.3 at that rate).
//
// Roles of a CTA's ten warps: TMA, MMA, eight of the epilogue (warp w reads the TMEM
// lane quarter w % 4 and one half of the columns).  A stage has two K steps of
// 64: a handshake costs about as much as a step's MMAs.  Two TMEM accumulators,
// so that a tile's epilogue runs beside the next one's MMAs.  Tiles are walked
// in bands of weight tiles (sched.cuh).
//
// The tensor core cuts what it adds to a sum off at the sum's last bits: one
// accumulator over K ends up 1.1e-9 K short of the exact sum, relative (measured:
// 2.1e-6 for K = 2048, 7.9e-6 for 7168).  That is nothing next to a bf16 output's
// 2^-9, but fp32 outputs would lose 3 of their bits by it: for these
// (LinearArgs::chunk) an accumulator sums 512 elements and the epilogue adds those
// sums in fp32 registers.  For bf16 outputs it sums all of K up to 65536 elements (7.2e-5,
// a 27th of the output's rounding), beyond that 32768 at a time: a weight gradient over 2^20
// rows would be 1.2e-3 short.
//
// SwiGLU: a tile's weight rows are BN / 2 gate rows and the up rows of the same
// columns, and an epilogue warp has both halves of its columns.
//
// Every mbarrier wait is bounded, as in the other GEMMs; LinearArgs::starve makes
// them run out for tests.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "bounds.cuh"
#include "internal.h"
#include "linear_epi.cuh"
#include "ptx.cuh"
#include "sched.cuh"

namespace moe {
namespace {

constexpr int kBK = 64;      // elements of a K step: 128 bytes of a row
constexpr int kSub = 2;      // K steps of a stage
constexpr int kUmmaK = 16;
constexpr int kBM = 128;     // rows of a CTA's tile
constexpr int kShortRows = 32;
constexpr int kMmaWarp = 1;
constexpr int kFirstEpi = 2;
constexpr int kEpiWarps = 8;
constexpr int kThreads = (kFirstEpi + kEpiWarps) * 32;
constexpr int kStageOutBytes = kEpiWarps * 4096;  // 32 x 32 sums per epilogue warp
constexpr int kChunkRows = kBK;                   // M/N-major: a box of 64 columns x 64 K
constexpr int kChunkBytes = kChunkRows * 128;
constexpr int kPartPitch = 64 + 4;                // split: floats of a row of partial sums
constexpr int kLongChunk = 32768 / kBK;           // K steps of an accumulator, bf16 and long K

template <int BN_>
struct Cfg {
  static constexpr int kABytes = kBM * 128;  // of a K step
  static constexpr int kBBytes = BN_ * 128;
  static constexpr int kStageBytes = kSub * (kABytes + kBBytes);
  static constexpr int kStages = 192 * 1024 / kStageBytes;
  // with A tiles of 32 rows
  static constexpr int kShortStages =
      192 * 1024 / (kSub * (kShortRows * 128 + kBBytes));
  static constexpr int kTmemCols = 2 * BN_;
  static constexpr int kCols = BN_ / 2;       // columns of an epilogue warp
  static constexpr int kSmemBytes = kStages * kStageBytes + kStageOutBytes + 1024;
};

// Operand tile descriptors of K step u, MMA k of a stage.
template <bool MN>
__device__ __forceinline__ uint64_t tile_desc(uint32_t addr) {
  return MN ? sw128_mnmajor_desc(addr, kChunkBytes) : sw128_kmajor_desc(addr);
}
template <bool MN>
constexpr uint32_t kMmaStep = MN ? kUmmaK * 128 : kUmmaK * 2;  // bytes

// The sums of a warp's 32 rows (a lane per row) and 32 columns go through `st`, 4 KB of
// shared memory of the warp, to lanes that have eight columns of a row, and on to the
// output.  16-byte pieces are placed so that a quarter warp meets no bank twice on the
// way in.
__device__ __forceinline__ void stage_rows(const uint32_t (&v)[32], uint4* st, int lane) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    st[lane * 8 + (i ^ (lane & 7))] =
        make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
}
// Rows [row0, row0 + rows), columns from col0 on.  SwiGLU: 16 columns, the gate's sums
// then the up's.  ROWS of a lane's (four or two) rows at once.
template <int ROWS = 4>
__device__ __forceinline__ void finish_rows(const LinearEpi& e, long long row0, int rows, int col0,
                                            const uint4* st, int lane) {
  __syncwarp();
  auto piece = [&](int r, int i, float (&z)[8]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint4 q = st[r * 8 + ((i + h) ^ (r & 7))];
      z[4 * h] = __uint_as_float(q.x);
      z[4 * h + 1] = __uint_as_float(q.y);
      z[4 * h + 2] = __uint_as_float(q.z);
      z[4 * h + 3] = __uint_as_float(q.w);
    }
  };
  if (e.act == MOE_LINEAR_SWIGLU) {
    constexpr int R = ROWS < 2 ? ROWS : 2;
    const int r0 = lane >> 1, p = lane & 1;  // rows r0 and r0 + 16
#pragma unroll
    for (int j = 0; j < 2; j += R) {
      float z[R][8], u[R][8];
      unsigned live = 0;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int r = r0 + 16 * (j + i);
        piece(r, 2 * p, z[i]);
        piece(r, 4 + 2 * p, u[i]);
        if (r < rows) live |= 1u << i;
      }
      finish8<true, R>(e, row0 + r0 + 16 * j, 16, live, col0 + 8 * p, z, u);
    }
  } else {
    const int r0 = lane >> 2, p = lane & 3;  // rows r0, r0 + 8, r0 + 16, r0 + 24
#pragma unroll
    for (int j = 0; j < 4; j += ROWS) {
      float z[ROWS][8], u[1][8];
      unsigned live = 0;
#pragma unroll
      for (int i = 0; i < ROWS; ++i) {
        const int r = r0 + 8 * (j + i);
        piece(r, 2 * p, z[i]);
        if (r < rows) live |= 1u << i;
      }
      finish8<false, ROWS>(e, row0 + r0 + 8 * j, 8, live, col0 + 8 * p, z, u);
    }
  }
  __syncwarp();
}

template <int BN, bool SPLIT, bool AMN, bool BMN>
__global__ void __launch_bounds__(kThreads, 1)
    linear_kernel(const __grid_constant__ LinearArgs a, const __grid_constant__ CUtensorMap tmA,
                  const __grid_constant__ CUtensorMap tmB) {
  using C = Cfg<BN>;
  extern __shared__ uint8_t smem_raw[];
  constexpr int kMaxStages = AMN ? C::kStages : C::kShortStages;
  __shared__ __align__(8) uint64_t full_bar[kMaxStages];
  __shared__ __align__(8) uint64_t empty_bar[kMaxStages];
  __shared__ __align__(8) uint64_t accf_bar[2];
  __shared__ __align__(8) uint64_t acce_bar[2];
  __shared__ __align__(8) uint64_t drain_bar;
  __shared__ uint32_t s_tmem_base;
  __shared__ int s_skip;
  __shared__ volatile int s_abort;
  __shared__ volatile int s_cluster_abort;  // split: some CTA of the cluster gave up

  // through a shuffle, so that the compiler knows it to be the same for a warp
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;
  const uint32_t rank = SPLIT ? cluster_ctarank() : 0u;
  const uint32_t smemA = (smem_u32(smem_raw) + 1023u) & ~1023u;
  // A K step is on its way for 1.3 us or so, and a CTA's rate is what it has on its
  // way in that time: with few rows, whose A tiles are short, twice as many stages.
  const bool short_a = !AMN && a.short_a;
  const uint32_t stages = short_a ? kMaxStages : C::kStages;
  const uint32_t a_bytes = short_a ? kShortRows * 128 : C::kABytes;
  const uint32_t smemB = smemA + stages * kSub * a_bytes;
  uint8_t* smem_gen = smem_raw + (smemA - smem_u32(smem_raw));
  uint4* out_stage = reinterpret_cast<uint4*>(smem_gen + C::kStages * C::kStageBytes);

  // what needs no input comes before the wait for the earlier kernels
  if (threadIdx.x == 0) {
    s_abort = 0;
    s_cluster_abort = 0;
    for (uint32_t i = 0; i < stages; ++i) {
      mbar_init(smem_u32(&full_bar[i]), 1);
      mbar_init(smem_u32(&empty_bar[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&accf_bar[i]), 1);
      mbar_init(smem_u32(&acce_bar[i]), kEpiWarps);
    }
    mbar_init(smem_u32(&drain_bar), 1);
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  if (warp == kMmaWarp) tmem_alloc(smem_u32(&s_tmem_base), C::kTmemCols);
  pdl_wait();
  pdl_launch_dependents();
  if (threadIdx.x == 0)
    s_skip = (a.status != nullptr && *reinterpret_cast<volatile int32_t*>(a.status) != 0);
  tc_fence_before_sync();
  if constexpr (SPLIT) {
    cluster_sync();
  } else {
    __syncthreads();
  }
  tc_fence_after_sync();
  // one answer per cluster: the status word may change while its CTAs start
  const bool skip = (SPLIT ? static_cast<int>(ld_shared_cluster_u32(
                                 mapa_shared(smem_u32(&s_skip), 0)))
                           : s_skip) != 0;
  const uint32_t tmem_base = s_tmem_base;

  const TileOrder order(a.m_tiles, a);
  const int total = skip ? 0 : a.m_tiles * a.n_tiles;
  const int csize = SPLIT ? a.splits : 1;
  const int first = blockIdx.x / csize;
  const int step = gridDim.x / csize;
  // this CTA's K steps
  const int kb = SPLIT ? a.k_steps * static_cast<int>(rank) / a.splits : 0;
  const int ke = SPLIT ? a.k_steps * (static_cast<int>(rank) + 1) / a.splits : a.k_steps;
  const uint64_t to = a.timeout_ns;
  const bool gated = a.epi.act == MOE_LINEAR_SWIGLU;

  // what this thread may leave in flight when a wait runs out in another warp
  unsigned issued = 0;
  bool issuer = false;

  if (warp == 0) {
    // ------------------------------------------------------- TMA producer
    if (elect_one() && !a.starve) {
      uint32_t stage = 0, phase = 0;
      bool ok = true;
      for (int tile = first; tile < total && ok; tile += step) {
        const Tile t = order(tile);
        const int m0 = t.mb * kBM;
        const int n0 = t.nt * (gated ? BN / 2 : BN);
        for (int kt = kb; kt < ke; kt += kSub) {
          if (!mbar_wait_suspend(smem_u32(&empty_bar[stage]), phase ^ 1, &s_abort, to)) {
            ok = false;
            break;
          }
          const uint32_t fb = smem_u32(&full_bar[stage]);
          const int nk = min(kSub, ke - kt);
          mbar_arrive_expect_tx(fb, (a_bytes + C::kBBytes) * nk);
          for (int u = 0; u < nk; ++u) {
            const uint32_t da = smemA + (stage * kSub + u) * a_bytes;
            const uint32_t db = smemB + (stage * kSub + u) * C::kBBytes;
            // coordinates along a row are in bytes (byte maps)
            if constexpr (AMN) {
#pragma unroll
              for (int c = 0; c < kBM / 64; ++c)
                tma_load_2d(da + c * kChunkBytes, &tmA, fb, (m0 + 64 * c) * 2, (kt + u) * kBK);
            } else {
              tma_load_2d(da, &tmA, fb, (kt + u) * 128, m0);
            }
            if constexpr (BMN) {
#pragma unroll
              for (int c = 0; c < BN / 64; ++c)
                tma_load_2d(db + c * kChunkBytes, &tmB, fb, (n0 + 64 * c) * 2, (kt + u) * kBK);
            } else if (gated) {  // boxes of BN / 2 rows
              tma_load_2d(db, &tmB, fb, (kt + u) * 128, n0);
              tma_load_2d(db + C::kBBytes / 2, &tmB, fb, (kt + u) * 128, a.epi.cols + n0);
            } else {
              tma_load_2d(db, &tmB, fb, (kt + u) * 128, n0);
            }
          }
          ++issued;
          if (++stage == stages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // --------------------------------------------------------- MMA issuer
    if (elect_one()) {
      // stage 0's descriptors; their address field counts 16 bytes
      const uint64_t a_desc0 = tile_desc<AMN>(smemA), b_desc0 = tile_desc<BMN>(smemB);
      uint32_t stage = 0, phase = 0, buf = 0, buf_phase = 0;
      bool ok = true;
      issuer = true;
      for (int tile = first; tile < total && ok; tile += step) {
        const Tile t = order(tile);
        // columns past the last one are left out of the MMA, in steps of 16
        const int n = gated ? BN : min(BN, (a.N - t.nt * BN + 15) & ~15);
        const uint32_t idesc = make_idesc_bf16(kBM, n, AMN, BMN);
        for (int k0 = kb; k0 < ke && ok; k0 += a.chunk) {
          const int kend = min(k0 + a.chunk, ke);
          if (!mbar_wait_suspend(smem_u32(&acce_bar[buf]), buf_phase ^ 1, &s_abort, to)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint32_t d_tmem = tmem_base + buf * BN;
          for (int kt = k0; kt < kend; kt += kSub) {
            if (!mbar_wait_suspend(smem_u32(&full_bar[stage]), phase, &s_abort, to)) {
              ok = false;
              break;
            }
            tc_fence_after_sync();
            const uint64_t ad = a_desc0 + stage * (kSub * a_bytes >> 4);
            const uint64_t bd = b_desc0 + stage * (kSub * C::kBBytes >> 4);
            auto mma = [&](int u) {
#pragma unroll
              for (int k = 0; k < kBK / kUmmaK; ++k)
                umma_bf16(d_tmem, ad + ((u * a_bytes + k * kMmaStep<AMN>) >> 4),
                          bd + ((u * C::kBBytes + k * kMmaStep<BMN>) >> 4), idesc,
                          kt > k0 || u > 0 || k > 0 ? 1u : 0u);
            };
            mma(0);
            if (kt + 1 < kend) mma(1);
            umma_commit(smem_u32(&empty_bar[stage]));
            if (++stage == stages) {
              stage = 0;
              phase ^= 1;
            }
          }
          if (!ok) break;
          umma_commit(smem_u32(&accf_bar[buf]));
          buf ^= 1;
          if (buf == 0) buf_phase ^= 1;
        }
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;
    const int half = (warp - kFirstEpi) >> 2;
    // where the two pieces of this warp's columns lie in the accumulator
    constexpr int kPiece = BN / 4;
    const int piece0 = half * (gated ? kPiece : C::kCols);
    const int piece1 = piece0 + (gated ? BN / 2 : kPiece);
    uint4* st = out_stage + (warp - kFirstEpi) * 256;
    uint32_t buf = 0, phase = 0;
    for (int tile = first; tile < total; tile += step) {
      const Tile t = order(tile);
      const long long row0 = static_cast<long long>(t.mb) * kBM + q * 32;
      const int rows = static_cast<int>(min(32ll, a.M - row0));
      const int col = gated ? t.nt * (BN / 2) + half * kPiece : t.nt * BN + half * C::kCols;
      // warps without a row or a column of the output only keep the barriers
      const bool live = rows > 0 && col < a.epi.cols;
      float acc[2 * kPiece];
#pragma unroll
      for (int i = 0; i < 2 * kPiece; ++i) acc[i] = 0.0f;
      // After a wait that ran out the tile's loop goes on to its end without
      // waiting, so that the warp stays converged; nothing is stored then.
      for (int k0 = kb; k0 < ke; k0 += a.chunk) {
        mbar_wait_suspend(smem_u32(&accf_bar[buf]), phase, &s_abort, to);
        __syncwarp();
        tc_fence_after_sync();
        if (live) {
          const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + buf * BN;
          uint32_t v[32], w[32];
          if constexpr (kPiece == 32) {
            tmem_ld32(taddr + piece0, v);
            tmem_ld32(taddr + piece1, w);
          } else {
            tmem_ld16<0>(taddr + piece0, v);
            tmem_ld16<16>(taddr + piece1, v);
          }
          tmem_wait_ld32(v);
          if constexpr (kPiece == 32) tmem_wait_ld32(w);
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            acc[i] += __uint_as_float(v[i]);
            if constexpr (kPiece == 32) acc[32 + i] += __uint_as_float(w[i]);
          }
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&acce_bar[buf]));
        buf ^= 1;
        if (buf == 0) phase ^= 1;
      }
      // one answer for the warp, whose lanes store together
      if (__any_sync(0xffffffffu, s_abort)) break;
      if (!live) continue;
      if constexpr (SPLIT) {
        // partial sums over the stages (all read by now)
        float* part = reinterpret_cast<float*>(smem_gen) + (q * 32 + lane) * kPartPitch;
        if (lane < rows) {
#pragma unroll
          for (int i = 0; i < kPiece; i += 4) {
            *reinterpret_cast<float4*>(part + piece0 + i) =
                make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
            *reinterpret_cast<float4*>(part + piece1 + i) =
                make_float4(acc[kPiece + i], acc[kPiece + i + 1], acc[kPiece + i + 2],
                            acc[kPiece + i + 3]);
          }
        }
      } else {
        uint32_t v[32];
#pragma unroll
        for (int s = 0; s < 2 * kPiece / 32; ++s) {
          if (gated) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              v[i] = __float_as_uint(acc[16 * s + i]);
              v[16 + i] = __float_as_uint(acc[kPiece + 16 * s + i]);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(acc[32 * s + i]);
          }
          stage_rows(v, st, lane);
          finish_rows(a.epi, row0, rows, col + s * (gated ? 16 : 32), st, lane);
        }
      }
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if (s_abort) {
    // no warp waits any more, and only these threads know what is under way
    if (issuer) {
      umma_commit(smem_u32(&drain_bar));
      drain_wait(smem_u32(&drain_bar), 0, to / 4);
    }
    const unsigned n0 = issued > stages ? issued - stages : 0;
    for (unsigned n = n0; n < issued; ++n)
      drain_wait(smem_u32(&full_bar[n % stages]), (n / stages) & 1, to / 4);
    __syncwarp();
  }
  if constexpr (SPLIT) {
    // a CTA that gave up has no sums to add: none of its cluster stores
    if (s_abort && threadIdx.x < a.splits)
      st_shared_cluster_u32(
          mapa_shared(smem_u32(const_cast<int*>(&s_cluster_abort)), threadIdx.x), 1u);
    __syncwarp();
    cluster_sync();
    // the cluster's tile: each CTA adds up and finishes its share of the rows,
    // the partial sums in rank order, eight columns to a thread
    if (first < total && !s_cluster_abort) {
      const Tile t = order(first);
      const int row0 = t.mb * kBM;
      const int rows = min(kBM, a.M - row0);
      const int r0 = rows * static_cast<int>(rank) / a.splits;
      const int r1 = rows * (static_cast<int>(rank) + 1) / a.splits;
      const int lg = gated ? 2 : 3;  // groups of eight columns: BN / 16 or BN / 8
      const int col0 = t.nt * (gated ? BN / 2 : BN);
      static_assert(BN == 64, "lg");
      for (int i = threadIdx.x; i < (r1 - r0) << lg; i += blockDim.x) {
        const int m = r0 + (i >> lg), c = 8 * (i & ((1 << lg) - 1));
        if (col0 + c >= a.epi.cols) continue;
        auto sums = [&](int at, float(&z)[8]) {
          const uint32_t addr = smemA + 4u * (m * kPartPitch + at);
#pragma unroll
          for (int j = 0; j < 8; ++j) z[j] = 0.0f;
          for (int p = 0; p < a.splits; ++p) {
            const uint32_t peer = mapa_shared(addr, p);
            const float4 x = ld_shared_cluster_f4(peer), y = ld_shared_cluster_f4(peer + 16);
            z[0] += x.x, z[1] += x.y, z[2] += x.z, z[3] += x.w;
            z[4] += y.x, z[5] += y.y, z[6] += y.z, z[7] += y.w;
          }
        };
        float z[1][8], u[1][8];
        sums(c, z[0]);
        if (gated) {
          sums(BN / 2 + c, u[0]);
          finish8<true, 1>(a.epi, static_cast<long long>(row0) + m, 0, 1u, col0 + c, z, u);
        } else {
          finish8<false, 1>(a.epi, static_cast<long long>(row0) + m, 0, 1u, col0 + c, z, u);
        }
      }
    }
    cluster_sync();  // the peers have read this CTA's shared memory
  }
  if (threadIdx.x == 0 && s_abort) report_error(a.status, MOE_ERR_TIMEOUT);
  if (warp == kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem_base, C::kTmemCols);
  }
}

// --------------------------------------------------------------- CTA pairs

// A tile of 256 x PN on a pair, PN 256 or 128, or (256, one accumulator) of fewer columns,
// LinearArgs::bn: each CTA has 128 rows of A and half of the B rows, and TMEM gets its 128
// rows x PN columns.  224 columns take 0.94 of 256's time (192 0.8, 160 no less) and fill
// 76 pairs better where 256 leave a round half empty: 4096 x 4096 x 4096 83 -> 78.5 us, 2048 x
// 4096 x 4096 44.7 -> 42.9, 1024 x 4096 x 7168 41.6 -> 40.2.  IN_REGS: the epilogue adds the
// accumulators' sums in fp32 registers (LinearArgs::chunk); otherwise a tile has one
// accumulator and is finished as it is read.  Both CTAs' copies complete on
// the leader's full barrier; the leader issues the MMAs and commits to both CTAs'
// barriers; the other CTA's epilogue gives its accumulator back through a
// barrier of its own CTA and a relaying lane (as in gemm_wpair.cu).  SwiGLU: the
// leader's B rows are gate rows, its peer's the up rows of the same columns.
template <int PN, bool IN_REGS, bool AMN, bool BMN>
__global__ void __launch_bounds__(kThreads, 1)
    linear_pair_kernel(const __grid_constant__ LinearArgs a, const __grid_constant__ CUtensorMap tmA,
                       const __grid_constant__ CUtensorMap tmB) {
  using P = Cfg<PN / 2>;  // a CTA's stages: 128 rows of A and PN / 2 of B per K step
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full_bar[P::kStages];
  __shared__ __align__(8) uint64_t empty_bar[P::kStages];
  __shared__ __align__(8) uint64_t accf_bar[2];
  __shared__ __align__(8) uint64_t acce_bar[2];
  __shared__ __align__(8) uint64_t relay_bar[2];
  __shared__ __align__(8) uint64_t drain_bar;
  __shared__ uint32_t s_tmem_base;
  __shared__ int s_skip;
  __shared__ volatile int s_abort;

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const uint32_t smemA = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t smemB = smemA + P::kStages * kSub * P::kABytes;
  uint8_t* smem_gen = smem_raw + (smemA - smem_u32(smem_raw));
  uint4* out_stage = reinterpret_cast<uint4*>(smem_gen + P::kStages * P::kStageBytes);

  if (threadIdx.x == 0) {
    s_abort = 0;
    for (int i = 0; i < P::kStages; ++i) {
      mbar_init(smem_u32(&full_bar[i]), 1);
      mbar_init(smem_u32(&empty_bar[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&accf_bar[i]), 1);
      mbar_init(smem_u32(&acce_bar[i]), kEpiWarps + 1);  // the leader's warps, the relay
      mbar_init(smem_u32(&relay_bar[i]), kEpiWarps);
    }
    mbar_init(smem_u32(&drain_bar), 1);
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  if (warp == kMmaWarp) tmem_alloc_pair(smem_u32(&s_tmem_base), 2 * PN);
  pdl_wait();
  pdl_launch_dependents();
  if (threadIdx.x == 0)
    s_skip = (a.status != nullptr && *reinterpret_cast<volatile int32_t*>(a.status) != 0);
  tc_fence_before_sync();
  cluster_sync();
  tc_fence_after_sync();
  const bool skip = ld_shared_cluster_u32(mapa_shared(smem_u32(&s_skip), 0)) != 0;
  const uint32_t tmem_base = s_tmem_base;

  const TileOrder order(a.m_tiles, a);
  const int total = skip ? 0 : a.m_tiles * a.n_tiles;
  const int first = blockIdx.x >> 1;
  const int step = gridDim.x >> 1;
  const uint64_t to = a.timeout_ns;
  const bool gated = a.epi.act == MOE_LINEAR_SWIGLU;
  const int bn = IN_REGS ? PN : a.bn;  // a multiple of 32
  // columns of tile nt's MMA: a multiple of 16
  auto tile_n = [&](int nt) {
    return gated ? bn : min(bn, (a.N - nt * bn + 15) & ~15);
  };
  unsigned issued = 0;
  bool issuer = false;

  if (warp == 0) {
    // ------------------------------------------------------- TMA producer
    if (elect_one() && !a.starve) {
      const uint32_t full0 = mapa_shared(smem_u32(&full_bar[0]), 0);
      uint32_t stage = 0, phase = 0;
      bool ok = true;
      for (int tile = first; tile < total && ok; tile += step) {
        const Tile t = order(tile);
        const int m0 = t.mb * 2 * kBM + static_cast<int>(rank) * kBM;
        const int n0 = gated ? t.nt * (bn / 2) + static_cast<int>(rank) * a.epi.cols
                             : t.nt * bn + static_cast<int>(rank) * (tile_n(t.nt) / 2);
        for (int kt = 0; kt < a.k_steps; kt += kSub) {
          if (!mbar_wait_suspend(smem_u32(&empty_bar[stage]), phase ^ 1, &s_abort, to)) {
            ok = false;
            break;
          }
          const uint32_t fb = full0 + stage * 8u;
          const int nk = min(kSub, a.k_steps - kt);
          // (boxes of 64 columns: all of them, also where a tile is narrower)
          const uint32_t b_bytes = BMN ? P::kBBytes : bn / 2 * 128;
          if (leader)
            mbar_arrive_expect_tx(smem_u32(&full_bar[stage]), 2u * (P::kABytes + b_bytes) * nk);
          for (int u = 0; u < nk; ++u) {
            const uint32_t da = smemA + (stage * kSub + u) * P::kABytes;
            const uint32_t db = smemB + (stage * kSub + u) * P::kBBytes;
            if constexpr (AMN) {
#pragma unroll
              for (int c = 0; c < 2; ++c)
                tma_load_2d_pair(da + c * kChunkBytes, &tmA, fb, (m0 + 64 * c) * 2, (kt + u) * kBK);
            } else {
              tma_load_2d_pair(da, &tmA, fb, (kt + u) * 128, m0);
            }
            if constexpr (BMN) {
#pragma unroll
              for (int c = 0; c < PN / 128; ++c)
                tma_load_2d_pair(db + c * kChunkBytes, &tmB, fb, (n0 + 64 * c) * 2, (kt + u) * kBK);
            } else {
              tma_load_2d_pair(db, &tmB, fb, (kt + u) * 128, n0);
            }
          }
          ++issued;
          if (++stage == P::kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // --------------------------------------------------------- MMA issuer
    if (leader && elect_one()) {
      const uint64_t a_desc0 = tile_desc<AMN>(smemA), b_desc0 = tile_desc<BMN>(smemB);
      uint32_t stage = 0, phase = 0, buf = 0, buf_phase = 0;
      bool ok = true;
      issuer = true;
      for (int tile = first; tile < total && ok; tile += step) {
        const Tile t = order(tile);
        const uint32_t idesc = make_idesc_bf16(2 * kBM, tile_n(t.nt), AMN, BMN);
        for (int k0 = 0; k0 < a.k_steps && ok; k0 += a.chunk) {
          const int kend = min(k0 + a.chunk, a.k_steps);
          if (!mbar_wait_bounded_cluster(smem_u32(&acce_bar[buf]), buf_phase ^ 1, &s_abort, to)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint32_t d_tmem = tmem_base + buf * PN;
          for (int kt = k0; kt < kend; kt += kSub) {
            if (!mbar_wait_bounded_cluster(smem_u32(&full_bar[stage]), phase, &s_abort, to)) {
              ok = false;
              break;
            }
            tc_fence_after_sync();
            const uint64_t ad = a_desc0 + stage * (kSub * P::kABytes >> 4);
            const uint64_t bd = b_desc0 + stage * (kSub * P::kBBytes >> 4);
            auto mma = [&](int u) {
#pragma unroll
              for (int k = 0; k < kBK / kUmmaK; ++k)
                umma_bf16_pair(d_tmem, ad + ((u * P::kABytes + k * kMmaStep<AMN>) >> 4),
                               bd + ((u * P::kBBytes + k * kMmaStep<BMN>) >> 4), idesc,
                               kt > k0 || u > 0 || k > 0 ? 1u : 0u);
            };
            mma(0);
            if (kt + 1 < kend) mma(1);
            umma_commit_pair(smem_u32(&empty_bar[stage]), 0x3);
            if (++stage == P::kStages) {
              stage = 0;
              phase ^= 1;
            }
          }
          if (!ok) break;
          umma_commit_pair(smem_u32(&accf_bar[buf]), 0x3);
          buf ^= 1;
          if (buf == 0) buf_phase ^= 1;
        }
      }
    } else if (!leader && lane == 0) {
      const uint32_t acce0 = mapa_shared(smem_u32(&acce_bar[0]), 0);
      uint32_t buf = 0, phase = 0;
      bool ok = true;
      for (int tile = first; tile < total && ok; tile += step) {
        for (int k0 = 0; k0 < a.k_steps; k0 += a.chunk) {
          if (!mbar_wait_suspend(smem_u32(&relay_bar[buf]), phase, &s_abort, to)) {
            ok = false;
            break;
          }
          mbar_arrive_cluster(acce0 + buf * 8u);
          buf ^= 1;
          if (buf == 0) phase ^= 1;
        }
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;
    const int half = (warp - kFirstEpi) >> 2;
    uint4* st = out_stage + (warp - kFirstEpi) * 256;
    constexpr int kPieces = PN / 64;  // of 32 columns, of an epilogue warp
    uint32_t buf = 0, phase = 0;
    auto wait = [&] {
      mbar_wait_suspend(smem_u32(&accf_bar[buf]), phase, &s_abort, to);
      __syncwarp();
      tc_fence_after_sync();
    };
    auto release = [&] {
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(leader ? smem_u32(&acce_bar[buf]) : smem_u32(&relay_bar[buf]));
      buf ^= 1;
      if (buf == 0) phase ^= 1;
    };
    for (int tile = first; tile < total; tile += step) {
      const Tile t = order(tile);
      const long long row0 =
          static_cast<long long>(t.mb) * 2 * kBM + static_cast<int>(rank) * kBM + q * 32;
      const int rows = static_cast<int>(max(0ll, min(32ll, a.M - row0)));
      // the second half of the warps has what the first, of PN / 2, leaves of the tile
      const int tile_cols = gated ? bn / 2 : bn;
      const int col0 = t.nt * tile_cols + half * (gated ? PN / 4 : PN / 2);
      const int end = min(a.epi.cols, (t.nt + 1) * tile_cols);
      const int width = gated ? 16 : 32;  // output columns of a step of the epilogue
      const bool live = rows > 0 && col0 < end;
      const uint32_t lanes = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
      uint32_t v[32];
      if constexpr (IN_REGS) {
        float acc[kPieces][32];
#pragma unroll
        for (int j = 0; j < kPieces; ++j)
#pragma unroll
          for (int i = 0; i < 32; ++i) acc[j][i] = 0.0f;
        // after a wait that ran out the loop goes on to its end without waiting, so
        // that the warp stays converged; nothing is stored then
        for (int k0 = 0; k0 < a.k_steps; k0 += a.chunk) {
          wait();
          if (live) {
#pragma unroll
            for (int j = 0; j < kPieces; ++j) {
              // SwiGLU: the first pieces are the gate's, the others the up's
              const int c = !gated             ? half * (PN / 2) + 32 * j
                            : j < kPieces / 2 ? half * (PN / 4) + 32 * j
                                              : PN / 2 + half * (PN / 4) + 32 * (j - kPieces / 2);
              // 128 sums and 32 more would not fit a thread's registers
#pragma unroll
              for (int h = 0; h < 32; h += 16) {
                tmem_ld16<0>(lanes + buf * PN + c + h, v);
                tmem_wait_ld16(v);
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[j][h + i] += __uint_as_float(v[i]);
              }
            }
          }
          release();
        }
        if (__any_sync(0xffffffffu, s_abort)) break;
        if (!live) continue;
#pragma unroll
        for (int s = 0; s < kPieces; ++s) {
          if (gated) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              v[i] = __float_as_uint(acc[s / 2][16 * (s & 1) + i]);
              v[16 + i] = __float_as_uint(acc[kPieces / 2 + s / 2][16 * (s & 1) + i]);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(acc[s][i]);
          }
          stage_rows(v, st, lane);
          finish_rows<PN == 256 ? 1 : 4>(a.epi, row0, rows, col0 + s * width, st, lane);
        }
      } else {
        wait();
        if (__any_sync(0xffffffffu, s_abort)) break;
        const int steps = !live ? 0 : min(kPieces, (end - col0 + width - 1) / width);
        for (int s = 0; s < steps; ++s) {
          if (gated) {
            tmem_ld16<0>(lanes + buf * PN + half * (PN / 4) + 16 * s, v);
            tmem_ld16<16>(lanes + buf * PN + bn / 2 + half * (PN / 4) + 16 * s, v);
          } else {
            tmem_ld32(lanes + buf * PN + half * (PN / 2) + 32 * s, v);
          }
          tmem_wait_ld32(v);
          stage_rows(v, st, lane);
          if (s + 1 == steps) release();  // the last sums are staged
          finish_rows(a.epi, row0, rows, col0 + s * width, st, lane);
        }
        if (steps == 0) release();
      }
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if (s_abort) {
    if (issuer) {
      umma_commit_pair(smem_u32(&drain_bar), 0x1);
      drain_wait(smem_u32(&drain_bar), 0, to / 4);
    }
    // the leader's barriers count both CTAs' copies; the other CTA, which cannot
    // wait on them, lets time pass
    if (issued > 0 && leader) {
      const unsigned n0 = issued > P::kStages ? issued - P::kStages : 0;
      for (unsigned n = n0; n < issued; ++n)
        drain_wait(smem_u32(&full_bar[n % P::kStages]), (n / P::kStages) & 1, to / 8);
    } else if (issued > 0) {
      const uint64_t t0 = global_timer_ns();
      while (global_timer_ns() - t0 < to / 8) {
      }
    }
    __syncwarp();
  }
  cluster_sync();
  if (threadIdx.x == 0 && s_abort) report_error(a.status, MOE_ERR_TIMEOUT);
  if (warp == kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc_pair(tmem_base, 2 * PN);
  }
}

// ------------------------------------------------------------------- launches

template <int BN, bool SPLIT, bool AMN, bool BMN>
cudaError_t prepare_one() {
  static std::atomic<unsigned long long> done{0};
  return allow_smem(linear_kernel<BN, SPLIT, AMN, BMN>, Cfg<BN>::kSmemBytes, done);
}

template <int PN, bool IN_REGS, bool AMN, bool BMN>
cudaError_t prepare_pair() {
  static std::atomic<unsigned long long> done{0};
  return allow_smem(linear_pair_kernel<PN, IN_REGS, AMN, BMN>, Cfg<PN / 2>::kSmemBytes, done);
}

int div_up(long long a, long long b) { return static_cast<int>((a + b - 1) / b); }

// Whether a tile has one accumulator for all of K.
bool one_accumulator(const LinearArgs& a) { return a.epi.out_bf16 && a.K <= kMostOfAccumulator; }

template <int BN, bool SPLIT, bool AMN, bool BMN>
cudaError_t launch_one(LinearArgs a, const LinearForm& f, const CUtensorMap& tmA,
                       const CUtensorMap& tmB, cudaStream_t s) {
  const cudaError_t err = prepare_one<BN, SPLIT, AMN, BMN>();
  if (err != cudaSuccess) return err;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = pdl_config(dim3(f.grid), dim3(kThreads), Cfg<BN>::kSmemBytes, s,
                                            attr, SPLIT ? f.splits : 1);
  return cudaLaunchKernelEx(&cfg, linear_kernel<BN, SPLIT, AMN, BMN>, a, tmA, tmB);
}

template <int PN, bool IN_REGS, bool AMN, bool BMN>
cudaError_t launch_pair(const LinearArgs& a, const LinearForm& f, const CUtensorMap& tmA,
                        const CUtensorMap& tmB, cudaStream_t s) {
  const cudaError_t err = prepare_pair<PN, IN_REGS, AMN, BMN>();
  if (err != cudaSuccess) return err;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg =
      pdl_config(dim3(f.grid), dim3(kThreads), Cfg<PN / 2>::kSmemBytes, s, attr, 2);
  return cudaLaunchKernelEx(&cfg, linear_pair_kernel<PN, IN_REGS, AMN, BMN>, a, tmA, tmB);
}

template <bool AMN, bool BMN>
cudaError_t launch_layout(const LinearArgs& a, const LinearForm& f, const CUtensorMap& tmA,
                          const CUtensorMap& tmB, cudaStream_t s) {
  if (f.pair && f.bn == 128)
    return launch_pair<128, true, AMN, BMN>(a, f, tmA, tmB, s);
  if (f.pair)
    return one_accumulator(a) ? launch_pair<256, false, AMN, BMN>(a, f, tmA, tmB, s)
                              : launch_pair<256, true, AMN, BMN>(a, f, tmA, tmB, s);
  if (f.splits > 1) return launch_one<64, true, AMN, BMN>(a, f, tmA, tmB, s);
  if (f.bn == 128) return launch_one<128, false, AMN, BMN>(a, f, tmA, tmB, s);
  return launch_one<64, false, AMN, BMN>(a, f, tmA, tmB, s);
}

}  // namespace

LinearHeld linear_held() {
  LinearHeld h = {};
  if (prepare_one<64, true, false, false>() != cudaSuccess ||
      prepare_pair<256, false, false, false>() != cudaSuccess) {
    cudaGetLastError();
    return h;
  }
  auto clusters = [](auto kern, int ctas, int smem) {
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg =
        pdl_config(dim3(ctas), dim3(kThreads), smem, nullptr, attr, ctas);
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
    return n;
  };
  for (int i = 0; i < 3; ++i)
    h.split[i] = clusters(linear_kernel<64, true, false, false>, 2 << i, Cfg<64>::kSmemBytes);
  h.pairs = clusters(linear_pair_kernel<256, false, false, false>, 2, Cfg<128>::kSmemBytes);
  return h;
}

// The form with the least estimated time: what a launch, its first loads and its last
// epilogue take, and rounds of tiles, each of them what its K steps take or what its
// epilogue does beside the next one's (GB300, us, operands from HBM; measured with the
// estimate in brackets).  333 x 2880 x 2880: 64 weight rows 11.8 (10.5), 128 16.0 (14.3),
// pairs of 128 14.4 (14.2); 512 x 4096 x 4096: 24.6 (23.8), 20.1 (18.5), 18.5 (17.6), pairs of
// 256 25.8 (25.2); 8192 x 4096 x 4096: 273 (280), 200 (203), 165 (169), 143 (135), pairs of 224
// 149 (146); 4096 x 4096 x 4096: 142 (147), 103 (104), 85 (88), 82 (80), 77 (77); 8192 x 7168
// x 256: 52 (51), 48 (47), 56 (56), 41 (43), 44 (46); 128 x 576 x 7168: 64 weight rows 20.9 (21.2), split
// by 2, 4, 8 14.8 (15.4), 11.0 (11.5), 10.3 (10.4).
LinearForm linear_form(const LinearArgs& a, int sms, const LinearHeld& held) {
  const bool gated = a.epi.act == MOE_LINEAR_SWIGLU;
  const int steps = div_up(a.K, kBK);
  LinearForm best = {};
  double least = 0.0;
  auto consider = [&](int bn, bool pair, int splits, long long slots, double step_us, double epi_us,
                      double base_us) {
    const long long n = static_cast<long long>(div_up(a.M, pair ? 256 : 128)) *
                        div_up(a.epi.cols, gated ? bn / 2 : bn);
    if (slots <= 0 || (splits > 1 && (n > slots || steps < 2 * splits))) return;
    const double us =
        base_us + div_up(n, slots) * std::max(step_us * div_up(steps, splits), epi_us);
    if (best.grid != 0 && us >= least) return;
    least = us;
    best.bn = bn;
    best.pair = pair;
    best.splits = splits;
    best.grid = static_cast<int>((splits > 1 ? n * splits : std::min(n, slots)) * (pair ? 2 : 1));
  };
  consider(64, false, 1, sms, 0.16, 1.0, 3.3);
  consider(128, false, 1, sms, 0.222, 1.8, 4.3);
  consider(128, true, 1, held.pairs, 0.182, 2.1, 6.0);
  consider(256, true, 1, held.pairs, 0.285, 3.0, 7.0);
  // the epilogue's first half of the warps has 128 columns of these too
  if (one_accumulator(a)) consider(224, true, 1, held.pairs, 0.272, 3.0, 7.0);
  for (int i = 0, s = 2; i < 3; ++i, s *= 2)
    consider(64, false, s, held.split[i], 0.16, 0.0, 5.8 + 0.3 * s);
  return best;
}

cudaError_t launch_linear(LinearArgs a, LinearLayout layout, const LinearForm& f,
                          const CUtensorMap& tmA, const CUtensorMap& tmB, cudaStream_t s) {
  const bool gated = a.epi.act == MOE_LINEAR_SWIGLU;
  const int bm = f.pair ? 2 * kBM : kBM;
  a.m_tiles = div_up(a.M, bm);
  a.n_tiles = div_up(a.epi.cols, gated ? f.bn / 2 : f.bn);
  a.bn = f.bn;
  a.band = std::min(a.n_tiles, f.bn > 128 ? 8 : 16);
  a.k_steps = div_up(a.K, kBK);
  a.chunk = !a.epi.out_bf16      ? 512 / kBK
            : one_accumulator(a) ? a.k_steps + (a.k_steps & 1)
                                 : kLongChunk;
  a.splits = f.splits;
  switch (layout) {
    case kRowsRows:
      return launch_layout<false, false>(a, f, tmA, tmB, s);
    case kRowsCols:
      return launch_layout<false, true>(a, f, tmA, tmB, s);
    default:
      return launch_layout<true, true>(a, f, tmA, tmB, s);
  }
}

}  // namespace moe
