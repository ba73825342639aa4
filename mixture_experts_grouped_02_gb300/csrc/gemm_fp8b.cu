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
// scale is one register of the thread that owns the row (rows of a on the
// MMA's M side), and the columns of a thread have one weight scale, so this
// costs one packed fma.rn.f32x2 for two elements.
//
// Two forms of one kernel, a template over the weight rows BN of a tile and
// the mode (fp8b_form chooses, with what each measured):
//  * kSingle: one CTA per tile of 128 rows x BN weight rows, 128 or 64;
//  * kSplit: a cluster of 2 to 8 CTAs shares one tile's K range and adds the
//    partial sums through distributed shared memory, in rank order, for
//    products with fewer tiles than SMs and a long K.
//
// Layout per CTA (one per SM, persistent, tiles walked in bands as in
// sched.cuh; kSplit: one tile per cluster):
//  * 192 KB of stages of two scale blocks each: A 2 x 128 rows x 128 bytes (32
//    rows when the row block has at most 32 valid rows), B 2 x BN rows,
//    128-byte swizzled, by TMA.  K past the tensor reads as zero codes.  Two
//    blocks to a stage because a handshake costs about as much as a block's
//    MMAs: a look at an mbarrier 55 clocks and more under load, a commit until
//    its waiters run 240;
//  * TMEM: two buffers of two fp32 blocks of BN columns; the columns past N
//    in the last tile are left out of the MMA's N;
//  * warp 0 TMA, warp 1 MMA, warp 2 the row scales (loaded by the threads
//    that need them they took 32 L1 lines per load and warp and held up the
//    buffers' release), warps 3-10 epilogue: warp w reads the lane quarter w %
//    4 and one half of the columns.  A warp whose 32 rows are all padding only
//    keeps the barriers.
//
// 8192 x 4096 x 7168: 197 us in a burst of 12 launches, 219 in a loop of seconds
// under the power cap (2.44 and 2.20 PFLOP/s; 1715 MHz, 375,000 clocks), about
// 840 clocks per stage of two scale blocks inside a tile and 2500 more per tile
// for its output.  What bounds a stage is shared memory: its MMAs need 512 clocks at the full rate and
// take them when the operands stay in place (all SMs busy), reading 64 KB at
// 128 bytes a clock; TMA's writes of the next 64 KB, at 256 bytes a clock, add
// to that.  The sum, 768, is what a stage takes when the epilogue only hands the
// buffers back (758; with 64 weight rows 576 and 560, with a quarter of A's
// bytes 672 and 676).  Fewer bytes per product need wider tiles.  Tried: 256
// columns with 16 epilogue warps, which spill at the 96 registers that so many
// threads leave (1,030,000 clocks), and 256 rows x 128 weight rows on CTA pairs
// (cta_group::2; 372,000 to 437,000 clocks with small changes elsewhere, at best
// 216 us where this form took 227), whose buffers come back 1060 clocks after
// their last MMA; pairs were left out as a second protocol for 5 %.  Not
// tried: 256 columns with 8 epilogue warps of 128 sums on registers that the
// other warps give up, and 256 x 256 pairs.  No gain from: a second issuing thread (414,000), 16 epilogue warps (420,000), buffers
// given back by scale block (384,000), four buffers of 64 columns, L2 copies of
// the weights ahead of the loads (393,000), outputs stored by TMA (384,000).
//
// Every mbarrier wait is bounded, as in the other GEMMs: a thread that gives
// up raises the CTA's abort flag, the copies and MMAs that any warp has in
// flight drain (with a limit), and the kernel records MOE_ERR_TIMEOUT and frees
// its TMEM.  Fp8bArgs::starve makes waits run out for tests of this path.
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "bounds.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "sched.cuh"

namespace moe {
namespace {

enum Mode { kSingle = 0, kSplit = 1 };  // Fp8bForm::mode

template <int BN_, int MODE>
struct Cfg {
  static constexpr int kBM = 128;
  static constexpr int kBK = 128;  // one scale block
  static constexpr int kSub = 2;   // scale blocks of a stage (two units of work)
  static constexpr int kUmmaK = 32;
  static constexpr int kABytes = kBM * kBK;
  static constexpr int kAShortRows = 32;
  static constexpr int kAShortBytes = kAShortRows * kBK;
  static constexpr int kBBytes = BN_ * kBK;
  static constexpr int kStageBytes = kSub * (kABytes + kBBytes);
  static constexpr int kStages = 192 * 1024 / kStageBytes;
  // buffers of kSub scale blocks: stage j waits for the epilogue of j - kBufs
  static constexpr int kBufs = 2;
  static constexpr int kBufCols = kSub * BN_;
  static constexpr int kTmemCols = kBufs * kBufCols;
  // Scale slots.  Stage j takes the slot of stage j - kSlots, which has been
  // read once the MMAs of stage j - kSlots + kBufs = j - kStages are done: they
  // wait for the buffer of j - kSlots, which every epilogue warp gives back by
  // an arrival that releases its lanes' reads of the slot.  With kStages slots,
  // the scales of a stage could be written only after the MMAs of the stage
  // before it: 249 us instead of 217 for 8192 x 4096 x 7168.
  static constexpr int kSlots = kStages + kBufs;
  static constexpr int kMmaWarp = 1;
  static constexpr int kScaleWarp = 2;
  static constexpr int kFirstEpi = 3;
  static constexpr int kEpiWarps = 8;
  static constexpr int kThreads = (kFirstEpi + kEpiWarps) * 32;
  static constexpr int kCols = BN_ / 2;  // columns of an epilogue thread
  static constexpr int kPartPitch = BN_ + 4;  // kSplit: floats of a row of partial sums
  static constexpr int kOutBytes = kEpiWarps * 2048;  // see store_rows
  static constexpr int kSmemBytes = kStages * kStageBytes + kOutBytes + 1024;
};

// A tile's rows: expert, first row, valid rows (0: none).
struct RowBlock {
  int e, r0, valid;
};

// Valid rows of part `sub` (128 rows each) of align block `bi`.
__device__ __forceinline__ int part_valid(const Fp8bArgs& a, const int4& bi, int sub) {
  if (!block_in_bounds(bi, a.E, a.cap, a.subs * 128, a.status)) return 0;
  return max(0, min(128, bi.w - 128 * sub));
}

// Row block `mb` of the call: 128 rows of a plain product, or part of an align
// block (blocks of 256 rows have two parts).
__device__ __forceinline__ RowBlock row_block(const Fp8bArgs& a, int mb) {
  RowBlock r;
  if (a.block_info == nullptr) {
    r.e = 0;
    r.r0 = mb * 128;
    r.valid = min(128, a.M - r.r0);
    return r;
  }
  const int b = mb / a.subs, sub = mb - b * a.subs;
  const int4 bi = reinterpret_cast<const int4*>(a.block_info)[b];
  r.e = bi.x;
  r.r0 = bi.z + 128 * sub;
  r.valid = part_valid(a, bi, sub);
  return r;
}

// Division by a divisor known once per launch, for tile indexes below 2^31.
// umulhi(x, floor((2^32 - 1) / d)) falls short of x / d by less than 2.
struct FastDiv {
  unsigned d, m;
  __device__ explicit FastDiv(unsigned d_) : d(d_), m(0xffffffffu / d_) {}
  __device__ __forceinline__ unsigned operator()(unsigned x) const {
    unsigned q = __umulhi(x, m);
    unsigned r = x - q * d;
    if (r >= d) ++q, r -= d;
    if (r >= d) ++q;
    return q;
  }
};

// decode_tile's order (sched.cuh; no K splits) without its divisions, which
// took the one thread that issues the MMAs about 1000 clocks a tile.
struct TileOrder {
  int num_blocks, n_tiles, band, full_bands;
  FastDiv by_band_tiles, by_band, by_tail;
  __device__ TileOrder(int blocks, const Fp8bArgs& a)
      : num_blocks(blocks),
        n_tiles(a.n_tiles),
        band(a.band),
        full_bands(a.n_tiles / a.band),
        by_band_tiles(static_cast<unsigned>(max(1, blocks * a.band))),
        by_band(static_cast<unsigned>(a.band)),
        by_tail(static_cast<unsigned>(max(1, a.n_tiles % a.band))) {}
  __device__ __forceinline__ Tile operator()(int tile) const {
    Tile t;
    t.split = 0;
    const int b = static_cast<int>(by_band_tiles(static_cast<unsigned>(tile)));
    const bool full = b < full_bands;
    const int nt0 = (full ? b : full_bands) * band;
    const unsigned w = static_cast<unsigned>(tile - nt0 * num_blocks);
    t.mb = static_cast<int>(full ? by_band(w) : by_tail(w));
    t.nt = nt0 + static_cast<int>(w) - t.mb * (full ? band : n_tiles - full_bands * band);
    return t;
  }
};

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

// Rows of any alignment: the sums of a warp's rows through `stage` (2 KB), 16
// columns at a time, so that lanes store consecutive elements of a row.  Out
// of line, as its registers would cost the main loop 5 to 15 % of its speed.
template <int COLS>
__device__ __noinline__ void store_rows_any(void* out, int N, int out_bf16, long long row0,
                                            int rows, int col, const float* acc, float* stage,
                                            int lane) {
  const int c = lane & 15;
  for (int c0 = 0; c0 < COLS && col + c0 < N; c0 += 16) {
    __syncwarp();
    // column-major pieces of 32 rows: neither side meets a bank twice
#pragma unroll
    for (int i = 0; i < 16; ++i) stage[i * 32 + ((lane + i) & 31)] = acc[c0 + i];
    __syncwarp();
    if (col + c0 + c < N) {
      for (int r = lane >> 4; r < rows; r += 2) {
        const float v = stage[c * 32 + ((r + c) & 31)];
        const long long o = (row0 + r) * N + col + c0 + c;
        if (out_bf16)
          static_cast<__nv_bfloat16*>(out)[o] = __float2bfloat16_rn(v);
        else
          static_cast<float*>(out)[o] = v;
      }
    }
  }
}

// The COLS sums of each of a warp's 32 rows (a lane per row) to columns
// [col, col + COLS) of out, those below N, for the first `rows` rows.  16-byte
// stores go through `stage`, 2 KB of shared memory of the warp: 64 bytes of
// every row at a time are written there by the row's lane, in 16-byte pieces
// rotated by the row so that neither side meets a bank twice, and read back
// four lanes to a row, so that a store covers 8 rows of 64 bytes instead of 32
// of 16.  (Stored straight from the rows' lanes, a tile's output kept the
// epilogue 3700 clocks from its next tile.)
template <int COLS>
__device__ __forceinline__ void store_rows(const Fp8bArgs& a, long long row0, int rows, int col,
                                           const uint64_t (&acc)[COLS / 2], uint4* stage,
                                           int lane) {
  const int n = min(COLS, a.N - col);
  const int es = a.out_bf16 ? 2 : 4;
  if (!a.wide_out) {
    float v[COLS];
#pragma unroll
    for (int i = 0; i < COLS / 2; ++i) unpack2(acc[i], v[2 * i], v[2 * i + 1]);
    store_rows_any<COLS>(a.out, a.N, a.out_bf16, row0, rows, col, v,
                         reinterpret_cast<float*>(stage), lane);
    return;
  }
  char* base = static_cast<char*>(a.out) + (row0 * a.N + col) * es;
  const long long pitch = static_cast<long long>(a.N) * es;
  const int rd_row = lane >> 2, piece = lane & 3;
  // 64 bytes of the rows from sum 16 c (fp32) or 32 c (bf16) on
  auto flush = [&](int c) {
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 8 * i + rd_row;
      const uint4 v = stage[4 * r + ((piece + (r >> 1)) & 3)];
      if (r < rows && (64 * c + 16 * piece) < n * es)
        *reinterpret_cast<uint4*>(base + r * pitch + 64 * c + 16 * piece) = v;
    }
    __syncwarp();
  };
  if (a.out_bf16) {
#pragma unroll
    for (int c = 0; c < COLS / 32; ++c) {
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        uint32_t p[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float lo, hi;
          unpack2(acc[16 * c + 4 * g + j], lo, hi);
          const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
          p[j] = *reinterpret_cast<const uint32_t*>(&h);
        }
        stage[4 * lane + ((g + (lane >> 1)) & 3)] = make_uint4(p[0], p[1], p[2], p[3]);
      }
      flush(c);
    }
  } else {
#pragma unroll
    for (int c = 0; c < COLS / 16; ++c) {
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        float v[4];
        unpack2(acc[8 * c + 2 * g], v[0], v[1]);
        unpack2(acc[8 * c + 2 * g + 1], v[2], v[3]);
        stage[4 * lane + ((g + (lane >> 1)) & 3)] =
            make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                       __float_as_uint(v[3]));
      }
      flush(c);
    }
  }
}

// Up to four consecutive elements of a row of out, the first `n` of them.
__device__ __forceinline__ void store4(const Fp8bArgs& a, long long o, int n, const float4& v) {
  if (a.out_bf16) {
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + o;
    const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
    if (a.wide_out) {
      *reinterpret_cast<uint2*>(out) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                                                  *reinterpret_cast<const uint32_t*>(&hi));
    } else {
      out[0] = lo.x;
      if (n > 1) out[1] = lo.y;
      if (n > 2) out[2] = hi.x;
      if (n > 3) out[3] = hi.y;
    }
  } else {
    float* out = static_cast<float*>(a.out) + o;
    if (a.wide_out) {
      *reinterpret_cast<float4*>(out) = v;
    } else {
      out[0] = v.x;
      if (n > 1) out[1] = v.y;
      if (n > 2) out[2] = v.z;
      if (n > 3) out[3] = v.w;
    }
  }
}

template <int BN, int MODE>
__global__ void __launch_bounds__(Cfg<BN, MODE>::kThreads, 1)
    fp8b_gemm_kernel(const __grid_constant__ Fp8bArgs a, const __grid_constant__ CUtensorMap tmA,
                     const __grid_constant__ CUtensorMap tmAShort,
                     const __grid_constant__ CUtensorMap tmB) {
  using C = Cfg<BN, MODE>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full_bar[C::kStages];
  __shared__ __align__(8) uint64_t empty_bar[C::kStages];
  __shared__ __align__(8) uint64_t acce_bar[C::kBufs];
  // sa * sb of the tile's rows for the scale blocks of a stage
  __shared__ float s_scale[C::kSlots][C::kSub][128];
  __shared__ __align__(8) uint64_t drain_bar;
  __shared__ uint32_t s_tmem_base;
  __shared__ int s_skip;
  __shared__ volatile int s_abort;
  __shared__ volatile int s_cluster_abort;  // kSplit: some CTA of the cluster gave up

  // through a shuffle, so that the compiler knows it to be the same for a warp
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;
  const uint32_t rank = MODE == kSingle ? 0u : cluster_ctarank();
  const uint32_t smemA = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t smemB = smemA + C::kStages * C::kSub * C::kABytes;
  uint8_t* smem_gen = smem_raw + (smemA - smem_u32(smem_raw));
  uint4* out_stage = reinterpret_cast<uint4*>(smem_gen + C::kStages * C::kStageBytes);

  pdl_wait();
  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    s_skip = (a.status != nullptr && *reinterpret_cast<volatile int32_t*>(a.status) != 0);
    s_abort = 0;
    s_cluster_abort = 0;
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(smem_u32(&full_bar[i]), 2);  // the expected bytes and the scales
      mbar_init(smem_u32(&empty_bar[i]), 1);
    }
    for (int i = 0; i < C::kBufs; ++i)
      mbar_init(smem_u32(&acce_bar[i]), C::kEpiWarps);
    mbar_init(smem_u32(&drain_bar), 1);
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if constexpr (MODE == kSingle) {
    __syncthreads();
  } else {
    cluster_sync();
  }
  // one answer per cluster: the status word may change while its CTAs start
  const bool skip =
      (MODE == kSingle ? s_skip
                       : static_cast<int>(ld_shared_cluster_u32(
                             mapa_shared(smem_u32(&s_skip), 0)))) != 0;
  if (!skip && warp == C::kMmaWarp) tmem_alloc(smem_u32(&s_tmem_base), C::kTmemCols);
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmAShort);
    tma_prefetch_desc(&tmB);
  }
  int num_blocks = 0;
  if (!skip)
    num_blocks = a.block_info == nullptr
                     ? a.max_blocks
                     : checked_num_blocks(*a.num_blocks, a.max_blocks, a.status) * a.subs;
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = s_tmem_base;

  const TileOrder order(num_blocks, a);
  const int total = num_blocks * a.n_tiles;
  const int csize = MODE == kSingle ? 1 : a.splits;
  const int first = blockIdx.x / csize;
  const int step = gridDim.x / csize;
  // this CTA's scale blocks
  const int kb = MODE == kSplit ? a.k_tiles * static_cast<int>(rank) / a.splits : 0;
  const int ke = MODE == kSplit ? a.k_tiles * (static_cast<int>(rank) + 1) / a.splits : a.k_tiles;
  const uint64_t to = a.timeout_ns;

  // what this thread may leave in flight (the producer's copies of stages, the
  // issuer's MMAs) when a wait runs out in another warp
  unsigned issued = 0;
  bool issuer = false;
  // the failure-path test: no copies, or no scales, so that waits run out
  const bool copies = a.starve == kStarveNone || a.starve == kStarveScales;
  const bool scales = a.starve == kStarveNone;

  // MMA columns of weight tile nt: a multiple of 16
  auto tile_cols = [&](int nt) { return min(BN, (a.N - nt * BN + 15) & ~15); };

  if (warp < C::kFirstEpi) {
    if (warp == 0) {
      // ----------------------------------------------------- TMA producer
      if (elect_one() && copies) {
        uint32_t stage = 0, phase = 0;
        bool ok = true;
        for (int tile = first; tile < total && ok; tile += step) {
          const Tile t = order(tile);
          const RowBlock r = row_block(a, t.mb);
          if (r.valid <= 0) continue;
          const bool short_a = r.valid <= C::kAShortRows;
          const CUtensorMap* map_a = short_a ? &tmAShort : &tmA;
          const uint32_t tx = C::kBBytes + (short_a ? C::kAShortBytes : C::kABytes);
          const int w_row = r.e * a.N + t.nt * BN;
          for (int kt = kb; kt < ke; kt += C::kSub) {
            if (!mbar_wait_suspend(smem_u32(&empty_bar[stage]), phase ^ 1, &s_abort, to)) {
              ok = false;
              break;
            }
            const uint32_t fb = smem_u32(&full_bar[stage]);
            const int nk = min(C::kSub, ke - kt);
            mbar_arrive_expect_tx(fb, tx * nk);
            for (int u = 0; u < nk; ++u) {
              const uint32_t da = smemA + (stage * C::kSub + u) * C::kABytes;
              const uint32_t db = smemB + (stage * C::kSub + u) * C::kBBytes;
              tma_load_2d(da, map_a, fb, (kt + u) * C::kBK, r.r0);
              tma_load_2d(db, &tmB, fb, (kt + u) * C::kBK, w_row);
            }
            ++issued;
            if (++stage == C::kStages) {
              stage = 0;
              phase ^= 1;
            }
          }
        }
      }
    } else if (warp == C::kMmaWarp && elect_one()) {
      // ----------------------------------------------------- MMA issuer
      // stage 0's descriptors; their address field counts 16 bytes
      const uint64_t a_desc0 = sw128_kmajor_desc(smemA), b_desc0 = sw128_kmajor_desc(smemB);
      uint32_t stage = 0, phase = 0, buf = 0, buf_phase = 0;
      bool ok = true;
      issuer = true;
      for (int tile = first; tile < total && ok; tile += step) {
        const Tile t = order(tile);
        if (row_block(a, t.mb).valid <= 0) continue;
        const uint32_t idesc = make_idesc(0, 128, tile_cols(t.nt));  // e4m3 x e4m3
        for (int kt = kb; kt < ke; kt += C::kSub) {
          // both looks in flight at once
          const uint32_t bf = smem_u32(&full_bar[stage]);
          const uint32_t be = smem_u32(&acce_bar[buf]);
          const bool rf = mbar_try_wait(bf, phase);
          const bool re = mbar_try_wait(be, buf_phase ^ 1);
          const uint32_t d_tmem = tmem_base + buf * C::kBufCols;
          const uint64_t ad = a_desc0 + stage * (C::kSub * C::kABytes >> 4);
          const uint64_t bd = b_desc0 + stage * (C::kSub * C::kBBytes >> 4);
          auto mma = [&](int u) {
#pragma unroll
            for (int k = 0; k < C::kBK / C::kUmmaK; ++k) {
              const uint64_t da = ad + u * (C::kABytes >> 4) + k * (C::kUmmaK >> 4);
              const uint64_t db = bd + u * (C::kBBytes >> 4) + k * (C::kUmmaK >> 4);
              umma_f8(d_tmem + u * BN, da, db, idesc, k > 0 ? 1u : 0u);
            }
          };
          if (!(rf || mbar_wait_suspended(bf, phase, &s_abort, to)) ||
              !(re || mbar_wait_suspended(be, buf_phase ^ 1, &s_abort, to))) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          mma(0);
          if (kt + 1 < ke) mma(1);
          // frees the stage and hands the buffer to the epilogue
          umma_commit(smem_u32(&empty_bar[stage]));
          if (++stage == C::kStages) {
            stage = 0;
            phase ^= 1;
          }
          if (++buf == C::kBufs) {
            buf = 0;
            buf_phase ^= 1;
          }
        }
      }
    } else if (warp == C::kScaleWarp && scales) {
      // ----------------------------------------------------- scales
      // A lane has four rows; the scale blocks of kGroup stages are loaded
      // together (a 32-byte sector of each row), while those of the kGroup
      // stages before them are written.
      constexpr int kGroup = 4, kBlocks = kGroup * C::kSub;
      // Rows that start on 16 bytes: four scale blocks to a load, 32 L1 lines for
      // four instead of one (8192 x 4096 x 7168: 371,000 clocks instead of 378,000).
      const bool wide = ((a.k_tiles | kb) & 3) == 0 &&
                        (reinterpret_cast<uintptr_t>(a.a_scale) & 15) == 0;
      uint32_t stage = 0, slot = 0;
      // The first kStages stages wait for nothing, the others for the MMAs of
      // stage j - kStages: for their slot, and so that the arrival below does
      // not come before the phase of the full barrier it counts in.
      int w_stage = 0;
      uint32_t w_phase = 0;
      int fresh = C::kStages;
      bool ok = true;
      for (int tile = first; tile < total && ok; tile += step) {
        const Tile t = order(tile);
        const RowBlock r = row_block(a, t.mb);
        if (r.valid <= 0) continue;
        const float* sb = a.w_scale + (static_cast<long long>(r.e) * a.n_scales +
                                       t.nt * BN / 128) * a.k_tiles;
        const float* sa = a.a_scale + (static_cast<long long>(r.r0) + lane) * a.k_tiles;
        const long long row32 = 32ll * a.k_tiles;
        float na[kBlocks][4], nb[kBlocks];
        auto load = [&](int kt) {
          if (wide) {
#pragma unroll
            for (int h = 0; h < kBlocks; h += 4) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float4 v =
                    kt + h < ke && lane + 32 * i < r.valid
                        ? __ldg(reinterpret_cast<const float4*>(sa + i * row32 + kt + h))
                        : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                na[h][i] = v.x, na[h + 1][i] = v.y, na[h + 2][i] = v.z, na[h + 3][i] = v.w;
              }
            }
          } else {
#pragma unroll
            for (int u = 0; u < kBlocks; ++u)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                na[u][i] = kt + u < ke && lane + 32 * i < r.valid ? __ldg(sa + i * row32 + kt + u)
                                                                  : 0.0f;
          }
#pragma unroll
          for (int u = 0; u < kBlocks; ++u) nb[u] = kt + u < ke ? __ldg(sb + kt + u) : 0.0f;
        };
        load(kb);
        for (int k0 = kb; k0 < ke && ok; k0 += kBlocks) {
          float s[kBlocks][4];
#pragma unroll
          for (int u = 0; u < kBlocks; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[u][i] = na[u][i] * nb[u];
          load(k0 + kBlocks);
#pragma unroll
          for (int g = 0; g < kGroup; ++g) {
            if (k0 + g * C::kSub >= ke || !ok) break;
            if (fresh > 0) {
              --fresh;
            } else {
              const int good =
                  mbar_wait_suspend(smem_u32(&empty_bar[w_stage]), w_phase, &s_abort, to);
              if (!__all_sync(0xffffffffu, good)) {
                ok = false;
                break;
              }
              if (++w_stage == C::kStages) {
                w_stage = 0;
                w_phase ^= 1;
              }
            }
#pragma unroll
            for (int u = 0; u < C::kSub; ++u)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                s_scale[slot][u][32 * i + lane] = s[g * C::kSub + u][i];
            // the slot joins its stage's full barrier: whoever sees that
            // stage's MMAs done sees it too
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&full_bar[stage]));
            if (++stage == C::kStages) stage = 0;
            if (++slot == C::kSlots) slot = 0;
          }
        }
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;
    const int col_in_tile = ((warp - C::kFirstEpi) >> 2) * C::kCols;
    uint32_t buf = 0, stage = 0, phase = 0, slot = 0;
    for (int tile = first; tile < total; tile += step) {
      const Tile t = order(tile);
      const RowBlock r = row_block(a, t.mb);
      if (r.valid <= 0) continue;
      const int local = q * 32 + lane;
      const int col = t.nt * BN + col_in_tile;
      // warps without a row or a column of the output only keep the barriers
      const bool live = q * 32 < r.valid && col < a.N;
      uint64_t acc[C::kCols / 2];
#pragma unroll
      for (int i = 0; i < C::kCols / 2; ++i) acc[i] = 0;
      // Waits for a stage's MMAs: its products are in TMEM.  After a wait that
      // ran out the tile's loop goes on to its end without waiting, so that the
      // warp stays converged; nothing is stored then.
      auto wait = [&] {
        mbar_wait_suspend(smem_u32(&empty_bar[stage]), phase, &s_abort, to);
        __syncwarp();
        tc_fence_after_sync();
      };
      // Gives the buffer and the scale slot back: the fence orders the TMEM
      // loads, the warp barrier and the arrival's release the lanes' reads of
      // s_scale, before the slot is written again.
      auto release = [&] {
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&acce_bar[buf]));
      };
      auto next_stage = [&] {
        buf ^= 1;
        if (++slot == C::kSlots) slot = 0;
        if (++stage == C::kStages) {
          stage = 0;
          phase ^= 1;
        }
      };
      if (!live) {
        for (int kt = kb; kt < ke; kt += C::kSub) {
          wait();
          release();
          next_stage();
        }
      } else if (kb < ke) {
        // Chunks of 32 columns: one is added while another one loads.  A load
        // takes about 110 clocks, an addition of 16 packed FMAs about 100 with
        // two warps per scheduler.  The buffer goes back once its last chunk
        // is in registers.
        constexpr int kChunks = C::kCols / 32;
        uint32_t va[32], vb[32];
        uint64_t s2;
        auto load = [&](int u, int j, uint32_t(&v)[32]) {
          tmem_ld32(tmem_base + (static_cast<uint32_t>(q * 32) << 16) + buf * C::kBufCols +
                        u * BN + col_in_tile + 32 * j,
                    v);
        };
        auto scale = [&](int u) {
          const uint32_t s = __float_as_uint(s_scale[slot][u][local]);
          s2 = pack2(s, s);
        };
        auto add = [&](int j, const uint32_t(&v)[32]) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            acc[16 * j + i] = fma2(pack2(v[2 * i], v[2 * i + 1]), s2, acc[16 * j + i]);
        };
        if constexpr (kChunks == 2) {
          wait();
          scale(0);
          load(0, 0, va);
          for (int kt = kb; kt < ke; kt += C::kSub) {
            tmem_wait_ld32(va);
            load(0, 1, vb);
            add(0, va);
            tmem_wait_ld32(vb);
            if (kt + 1 < ke) {
              load(1, 0, va);
              add(1, vb);
              scale(1);
              tmem_wait_ld32(va);
              load(1, 1, vb);
              add(0, va);
              tmem_wait_ld32(vb);
            }
            release();
            next_stage();
            if (kt + C::kSub < ke) {
              wait();
              load(0, 0, va);
            }
            add(1, vb);
            if (kt + C::kSub < ke) scale(0);
          }
        } else {
          for (int kt = kb; kt < ke; kt += C::kSub) {
            wait();
            scale(0);
            load(0, 0, va);
            tmem_wait_ld32(va);
            if (kt + 1 < ke) {
              add(0, va);
              scale(1);
              load(1, 0, va);
              tmem_wait_ld32(va);
            }
            release();
            add(0, va);
            next_stage();
          }
        }
      }
      // A wait ran out: no output, and no further tile.  One answer for the
      // warp, whose lanes store together (another thread may raise the flag
      // between two lanes' reads of it).
      if (__any_sync(0xffffffffu, s_abort)) break;
      if constexpr (MODE == kSplit) {
        // partial sums over the stages (all read by now), a row's kPartPitch
        // floats apart so that neither side of the exchange meets a bank twice
        float4* part = reinterpret_cast<float4*>(reinterpret_cast<float*>(smem_gen) +
                                                 local * C::kPartPitch + col_in_tile);
        if (live && local < r.valid) {
#pragma unroll
          for (int i = 0; i < C::kCols / 4; ++i) {
            float4 v;
            unpack2(acc[2 * i], v.x, v.y);
            unpack2(acc[2 * i + 1], v.z, v.w);
            part[i] = v;
          }
        }
      } else {
        if (live)
          store_rows<C::kCols>(a, r.r0 + q * 32, min(32, r.valid - q * 32), col, acc,
                               out_stage + (warp - C::kFirstEpi) * 128, lane);
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
    const unsigned n0 = issued > C::kStages ? issued - C::kStages : 0;
    for (unsigned n = n0; n < issued; ++n)
      drain_wait(smem_u32(&full_bar[n % C::kStages]), (n / C::kStages) & 1, to / 4);
    __syncwarp();
  }
  if constexpr (MODE == kSplit) {
    // a CTA that gave up has no sums to add: none of its cluster stores
    if (s_abort && threadIdx.x < a.splits)
      st_shared_cluster_u32(
          mapa_shared(smem_u32(const_cast<int*>(&s_cluster_abort)), threadIdx.x), 1u);
    __syncwarp();
    cluster_sync();
    // the cluster's tile: each CTA adds up and stores 64 / splits of its
    // columns, the partial sums in rank order, four columns to a thread
    if (first < total && !s_cluster_abort) {
      const Tile t = order(first);
      const RowBlock r = row_block(a, t.mb);
      const int lg = __ffs(BN / 4 / a.splits) - 1;  // splits is 2, 4 or 8
      const int c0 = static_cast<int>(rank) * (BN / a.splits);
      for (int i = threadIdx.x; i < r.valid << lg; i += blockDim.x) {
        const int c = c0 + 4 * (i & ((1 << lg) - 1)), m = i >> lg;
        const int col = t.nt * BN + c;
        if (col >= a.N) continue;
        const uint32_t at = smemA + 4u * (m * C::kPartPitch + c);
        float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int p = 0; p < a.splits; p += 2) {
          const float4 u = ld_shared_cluster_f4(mapa_shared(at, p));
          const float4 v = ld_shared_cluster_f4(mapa_shared(at, p + 1));
          sum.x = (sum.x + u.x) + v.x;
          sum.y = (sum.y + u.y) + v.y;
          sum.z = (sum.z + u.z) + v.z;
          sum.w = (sum.w + u.w) + v.w;
        }
        store4(a, static_cast<long long>(r.r0 + m) * a.N + col, a.N - col, sum);
      }
    }
    cluster_sync();  // the peers have read this CTA's shared memory
  }
  if (threadIdx.x == 0 && s_abort) report_error(a.status, MOE_ERR_TIMEOUT);
  if (!skip && warp == C::kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem_base, C::kTmemCols);
  }
}

template <int BN, int MODE>
cudaError_t prepare_kernel() {
  // once per device: the attribute outlives the launch
  static std::atomic<unsigned long long> done{0};
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  err = cudaFuncSetAttribute(fp8b_gemm_kernel<BN, MODE>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Cfg<BN, MODE>::kSmemBytes);
  if (err == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return err;
}

template <int BN, int MODE>
cudaError_t launch(Fp8bArgs a, const Fp8bForm& f, const Fp8bMaps& maps, cudaStream_t s) {
  using C = Cfg<BN, MODE>;
  cudaError_t err = prepare_kernel<BN, MODE>();
  if (err != cudaSuccess) return err;
  a.n_tiles = (a.N + BN - 1) / BN;
  // Tiles in flight together: 152 / 16 row blocks by 16 weight tiles.  In bands
  // of 4, 8, 16 and 32 weight tiles 8192 rows over 32 experts of 4096 x 7168 took
  // 302, 282, 276 and 278 us, 8192 x 4096 x 7168 210, 208, 205 and 206.
  a.band = std::min(a.n_tiles, 16);
  a.splits = f.splits;
  cudaLaunchAttribute attr[2];
  const unsigned cluster = MODE == kSplit ? f.splits : 1;
  const cudaLaunchConfig_t cfg =
      pdl_config(dim3(f.grid), dim3(C::kThreads), C::kSmemBytes, s, attr, cluster);
  return cudaLaunchKernelEx(&cfg, fp8b_gemm_kernel<BN, MODE>, a, maps.a, maps.a_short, maps.b);
}

long long div_up(long long a, long long b) { return (a + b - 1) / b; }

}  // namespace

// Clusters of 2, 4 and 8 CTAs of the split form the current device holds at
// once, 0 where unknown.
Fp8bHeld fp8b_held() {
  using C = Cfg<64, kSplit>;
  Fp8bHeld h = {};
  if (prepare_kernel<64, kSplit>() != cudaSuccess) {
    cudaGetLastError();
    return h;
  }
  for (int i = 0; i < 3; ++i) {
    const int ctas = 2 << i;
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg =
        pdl_config(dim3(ctas), dim3(C::kThreads), C::kSmemBytes, nullptr, attr, ctas);
    if (cudaOccupancyMaxActiveClusters(&h.split[i], fp8b_gemm_kernel<64, kSplit>, &cfg) !=
        cudaSuccess) {
      cudaGetLastError();
      h.split[i] = 0;
    }
  }
  return h;
}

// The form with the least estimated time: rounds of tiles times what a stage
// takes (GB300, us: 0.36 with 64 weight rows, 0.55 with 128; 8192 x 4096 x 7168
// takes 274 and 219 under the power cap).  Measured around the choice, operands
// from HBM: 333 x 2880 x 2880 in 8.6 us with 64 rows and 11.0 with 128; 1024 x
// 4096 x 7168 in 41 and 32; 8192 rows of 32 experts against 4096 x 7168 in 407
// and 296.  A sorted list's row blocks are
// estimated from its capacity: at least one row per align block and all but
// the padding of E blocks; half a block of padding per expert that has rows.
Fp8bForm fp8b_form(const Fp8bArgs& a, int sms, const Fp8bHeld& held) {
  Fp8bForm f;
  f.splits = 1;
  f.mode = kSingle;
  const long long n64 = div_up(a.N, 64), n128 = div_up(a.N, 128);
  const long long max_blocks = static_cast<long long>(a.max_blocks) * a.subs;
  double blocks = static_cast<double>(max_blocks);
  if (a.block_info != nullptr) {
    const long long rows =
        std::max<long long>(a.max_blocks, a.cap - static_cast<long long>(a.E) * (a.block_m - 1));
    const double experts = static_cast<double>(std::min<long long>(a.E, rows));
    blocks = std::min(blocks, static_cast<double>(rows) / std::min(128, a.block_m) + experts / 2);
  }
  const double us64 = 0.36 * std::ceil(blocks * n64 / sms);
  const double us128 = 0.55 * std::ceil(blocks * n128 / sms);
  if (us128 <= us64) {
    f.bn = 128;
    f.grid = static_cast<int>(std::min<long long>(sms, max_blocks * n128));
  } else {
    f.bn = 64;
    f.grid = static_cast<int>(std::min<long long>(sms, max_blocks * n64));
    // Splitting K by s, where all the clusters are resident at once: 0.29 us
    // for every stage a CTA has less, against 2 us of cluster launch and
    // barriers and 2.2 ns per row and partial sum to exchange them (operands from
    // HBM, 16 x 576 x 7168: 11.9 us whole, 9.6, 7.8 and 7.0 by 2, 4 and 8; 128 x
    // 576 x 7168: 12.7, 10.8, 9.3 and 9.7; 128 x 4096 x 7168: 13.8 whole, 12.7 by
    // 2; 16 x 2880 x 2880: 7.6 whole, 7.9 by 2; 333 x 1024 x 4096: 8.9 and 9.2).
    const int stages = (a.k_tiles + 1) / 2;
    const double rows = a.block_info != nullptr ? std::min(a.block_m, 128) : std::min(a.M, 128);
    double best = 0.0;
    for (int i = 0, s = 2; i < 3; ++i, s *= 2) {
      const double gain = 0.29 * (stages - div_up(stages, s)) - 2.0 - 0.0022 * rows * s;
      if (max_blocks * n64 <= held.split[i] && gain > best) {
        best = gain;
        f.mode = kSplit;
        f.splits = s;
        f.grid = static_cast<int>(max_blocks * n64 * s);
      }
    }
  }
  return f;
}

cudaError_t launch_fp8b_gemm(const Fp8bArgs& a, const Fp8bForm& f, const Fp8bMaps& maps,
                             cudaStream_t s) {
  if (f.mode == kSplit) return launch<64, kSplit>(a, f, maps, s);
  return f.bn == 128 ? launch<128, kSingle>(a, f, maps, s) : launch<64, kSingle>(a, f, maps, s);
}

}  // namespace moe
