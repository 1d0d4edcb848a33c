// Product of signed bytes with a scale per row of a (token) and per row of b
// (output channel) on the 5th-generation tensor cores, with the block's
// epilogues (the projections of the summary page's "Method" block update):
//
//   out[m][n] = epi(sa[m] sb[n] sum_k a[m][k] b[n][k] + bias[n])
//
// The sums are exact (int32 accumulators in TMEM, K < 131072: 2^17 products of -128 are
// 2^31); the scales, the bias and the epilogue are applied in fp32 and rounded once.
//
// Design: persistent warp-specialised kernel as for the bf16 product: TMA loads of
// 128-byte k-blocks (128-byte swizzle) through an mbarrier ring, one thread
// issuing tcgen05.mma kind::i8 (K = 32 per instruction, twice the bf16 rate), and
// epilogue warps that drain a double-buffered accumulator, stage blocks of 32 rows x
// 128 bytes in swizzled shared memory and leave them by TMA stores.
//   CG = 2: CTA pairs, 256 x 256 tiles (an SM reads its 128 rows of a and half of
//           the 256 columns of b): many rows.
//   CG = 1: one CTA, 128 x 64 tiles, so that a few hundred rows spread over the SMs;
//           with a long k and too few of them, a cluster of CTAs for each (below).
//   KEEP_B (pairs, k <= 512, where it gains: keeps_b): a pair stays in its 256 columns and
//           keeps their b in shared memory, which halves what L2 hands to the SMs.
// Measured on one B200, bursts of 20: 8192^3 at 2.9-3.1 P op/s, where the operands'
// way out of L2 (about 12 TB/s) bounds it (without b's loads 3.7); 131075 x 2048 x 512
// to f16 146 us (b reloaded: 152), its output's way to DRAM beside the epilogue (no
// stores: 105, no epilogue arithmetic: 139); to fp32 196 us, 5.8 TB/s. In a long run
// at the power limit the f16 one takes 170 us.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "common.cuh"
#include "ops.h"
#include "ptx.cuh"
#include "rowvec.cuh"
#include "tmap.h"

namespace mtgr {

namespace {

constexpr int BM = 128;   // rows of a per CTA
constexpr int BK = 128;   // bytes of k per stage: one swizzle row
constexpr int A_BYTES = BM * BK;
constexpr int kKeepK = 512;  // longest k whose tile of b stays in shared memory

template <int CG>
struct Shape {
  static constexpr int kBN = CG == 2 ? 256 : 64;   // columns of a tile
  static constexpr int kBRows = kBN / CG;          // rows of b per CTA
  static constexpr int kBBytes = kBRows * BK;
  static constexpr int kStageBytes = A_BYTES + kBBytes;
  static constexpr int kTileM = BM * CG;
  static constexpr int kTmemCols = 2 * kBN;
};

// The epilogue's split. A warp owns 32 rows (its TMEM lane quarter) and every
// (kWarps / 4)th share of the columns, in staging blocks of 32 rows x 128 bytes: whole
// lines for the TMA store. Sixteen warps for the 16-bit outputs of the pair form,
// whose main loop is short at K = 512; eight for its fp32 outputs.
template <int OUT, int CG, bool KEEP_B>
struct Epi {
  static constexpr int kWarps = CG == 2 ? (OUT != MTGR_F32 ? 16 : 8) : 4;
  static constexpr int kThreads = 64 + 32 * kWarps;
  static constexpr int kCols = OUT == MTGR_F32 ? 32 : 64;  // columns of a staging block
  static constexpr int kBlocks = (Shape<CG>::kBN / kCols) / (kWarps / 4);  // a warp's blocks per tile
  static constexpr int kBufs = kBlocks > 1 ? 2 : 1;
  static constexpr int kStg = 4096;
  static constexpr int kStages = KEEP_B || CG == 1 ? 6 : 5;
  static constexpr int kBBlocks = KEEP_B ? kKeepK / BK : kStages;  // blocks of b in shared memory
  static constexpr size_t kSmem = 1024 + (size_t)kStages * A_BYTES + (size_t)kBBlocks * Shape<CG>::kBBytes +
                                  (size_t)kWarps * kBufs * kStg + 256;
  static_assert(kSmem <= 227 * 1024, "shared memory of a block");
};

struct Args {
  int M, N, K;
  const float* sa;
  const float* sb;
  const float* bias;
  const float* resid;
  int q_cols;
  int32_t* status;
};

// Instruction descriptor of tcgen05.mma kind::i8: D int32 (2 at bits 4-5), A and
// B signed bytes (1 at 7-9 and 10-12), both K-major, N >> 3 at 17, M >> 4 at 24.
constexpr uint32_t idesc_i8(int M, int N) {
  return (2u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

template <int CG>
__device__ __forceinline__ void mma_i8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate) {
  if constexpr (CG == 2) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
  }
}

// 16-byte chunk c of row r of a staging block (128-byte rows, 128-byte swizzle)
__device__ __forceinline__ uint32_t stg_off(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }

// 32 columns' values of a per-column array (16-byte aligned), the same for every
// lane; columns past N (N % 8 == 0) are 0. FULL: there are none.
template <bool FULL>
__device__ __forceinline__ void load_cols(const float* p, int col0, int N, float4 (&v)[8]) {
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    if (FULL || col0 + 4 * c < N) v[c] = __ldg(reinterpret_cast<const float4*>(p + col0) + c);
    else v[c] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
}

// The scales, bias and epilogue of 32 columns [col0, col0 + 32) of one row whose
// TMEM load is under way: the column scales' loads run beside it, `loaded` when it
// is done. The result goes to chunks [c0, ...) of row r of the staging block. live: a row
// of the output; one behind the last is not stored and, of the bias alone, reports no range.
template <int EPI, int OUT, bool FULL, typename Loaded>
__device__ __forceinline__ void epilogue_cols(const Args& a, int col0, float sa, bool live, uint32_t (&acc)[32],
                                              const float4 (&res)[8], uint8_t* stg, int r, int c0,
                                              Loaded loaded) {
  float4 sb[8];
  load_cols<FULL>(a.sb, col0, a.N, sb);
  tmem_ld_wait();
  reg_fence(acc);
  loaded();
  float v[32];
  const f2 sa2 = both(sa);
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const float2 lo = unpair2(mul2(pair2(__int2float_rn((int)acc[4 * c]), __int2float_rn((int)acc[4 * c + 1])),
                                  mul2(sa2, pair2(sb[c].x, sb[c].y))));
    const float2 hi = unpair2(mul2(pair2(__int2float_rn((int)acc[4 * c + 2]), __int2float_rn((int)acc[4 * c + 3])),
                                  mul2(sa2, pair2(sb[c].z, sb[c].w))));
    v[4 * c] = lo.x; v[4 * c + 1] = lo.y; v[4 * c + 2] = hi.x; v[4 * c + 3] = hi.y;
  }
  if (a.bias != nullptr) {
    load_cols<FULL>(a.bias, col0, a.N, sb);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      v[4 * c] += sb[c].x; v[4 * c + 1] += sb[c].y; v[4 * c + 2] += sb[c].z; v[4 * c + 3] += sb[c].w;
    }
  }
  if (EPI == MTGR_EPI_SILU) {
    // v / (1 + e^-v), e^-v by __expf, within 2 + 1.2 |v| ulp (rows rounded to 8 bits are
    // off by far more): a tanh approximation would leave the small values of
    // negative v with only a few right bits. (One reciprocal for two values,
    // 1/a = b / (a b), measured 212 against 199 us at 131075 x 2048 x 512.)
#pragma unroll
    for (int c = 0; c < 32; ++c) v[c] = __fdividef(v[c], 1.0f + __expf(-v[c]));
  }
  if (EPI == MTGR_EPI_RESID) {
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      v[4 * c] += res[c].x; v[4 * c + 1] += res[c].y; v[4 * c + 2] += res[c].z; v[4 * c + 3] += res[c].w;
    }
  }
  if (col0 < a.q_cols) {
#pragma unroll
    for (int c = 0; c < 32; ++c) v[c] *= 0.5f;
  }
  if (OUT == MTGR_F32) {
#pragma unroll
    for (int c = 0; c < 8; ++c)
      *reinterpret_cast<float4*>(stg + stg_off(r, c0 + c)) =
          make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
  } else {
    uint32_t w[16];
#pragma unroll
    for (int k = 0; k < 16; ++k)
      w[k] = OUT == MTGR_F16 ? cvt_f16x2(v[2 * k], v[2 * k + 1]) : cvt_bf16x2(v[2 * k], v[2 * k + 1]);
#pragma unroll
    for (int c = 0; c < 4; ++c)
      *reinterpret_cast<uint4*>(stg + stg_off(r, c0 + c)) = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
    if (OUT == MTGR_F16) {
      // the conversion saturates: a value beyond f16 is reported. The largest
      // f16 among the results (two per instruction) tells whether one can be
      __half2 m = __habs2(*reinterpret_cast<__half2*>(&w[0]));
#pragma unroll
      for (int k = 1; k < 16; ++k) m = __hmax2(m, __habs2(*reinterpret_cast<__half2*>(&w[k])));
      const bool full = __half2float(__hmax(__low2half(m), __high2half(m))) >= 65504.f;
      if (__any_sync(0xffffffffu, full)) {
        float mx = 0.f;
#pragma unroll
        for (int c = 0; c < 32; ++c) mx = fmaxf(mx, fabsf(v[c]));
        if (live && mx > 65504.f) set_status(a.status, MTGR_ERR_RANGE);
      }
    }
  }
}

template <int EPI, int OUT, int CG, bool KEEP_B>
__global__ void __launch_bounds__(Epi<OUT, CG, KEEP_B>::kThreads, 1)
    gemm_i8_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const __grid_constant__ CUtensorMap tmO, Args args) {
  using S = Shape<CG>;
  using E = Epi<OUT, CG, KEEP_B>;
  constexpr int NST = E::kStages, BN = S::kBN;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + NST * A_BYTES;
  uint8_t* sStg = sB + E::kBBlocks * S::kBBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sStg + E::kWarps * E::kBufs * E::kStg);
  uint64_t* full = bars;
  uint64_t* empty = bars + NST;
  uint64_t* acc_full = bars + 2 * NST;
  uint64_t* acc_empty = bars + 2 * NST + 2;
  uint64_t* b_full = bars + 2 * NST + 4;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * NST + 5);

  const int warp = warp_id(), lane = lane_id();
  const int M = args.M, N = args.N;
  const int n_tiles = (N + BN - 1) / BN;
  const int m_tiles = (M + S::kTileM - 1) / S::kTileM;
  const int kblocks = (args.K + BK - 1) / BK;  // a ragged last block is zero-filled by the loads
  const uint32_t rank = CG == 2 ? cluster_ctarank() : 0u;
  const int unit = CG == 2 ? (int)(blockIdx.x >> 1) : (int)blockIdx.x;
  const int units = CG == 2 ? (int)(gridDim.x >> 1) : (int)gridDim.x;
  // The i-th tile of this block or pair; false behind the last. KEEP_B: it stays in
  // its columns (units >= n_tiles), whose b stays in shared memory, and takes every
  // so many-th row tile, as many as every other column's pairs, so that a row's tiles
  // are written at about the same time; else all tiles in turn, columns first.
  const auto tile_at = [&](int i, int& mb, int& nb) {
    if constexpr (KEEP_B) {
      const int per = units / n_tiles;  // pairs a column of tiles; the rest of the pairs have none
      nb = unit % n_tiles;
      mb = unit / n_tiles + i * per;
      return unit < per * n_tiles && mb < m_tiles;
    } else {
      const int t = unit + i * units;
      mb = t / n_tiles;
      nb = t - mb * n_tiles;
      return mb < m_tiles;
    }
  };

  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmO);
    for (int s = 0; s < NST; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&acc_full[a], 1);
      mbar_init(&acc_empty[a], CG * E::kWarps);  // the pair's epilogue warps, on the leader's barrier
    }
    mbar_init(b_full, 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    if constexpr (CG == 2) {
      tmem_alloc_cg2(tmem_slot, S::kTmemCols);
      tmem_relinquish_cg2();
    } else {
      tmem_alloc(tmem_slot, S::kTmemCols);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  if constexpr (CG == 2) cluster_sync();
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  bool timed_out = false;
  dependent_wait();  // a's bytes and scales may be another kernel's of the same call

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      int mb, nb;
      if (KEEP_B && tile_at(0, mb, nb)) {
        if (rank == 0) mbar_arrive_expect_tx(b_full, 2 * kblocks * S::kBBytes);
        const uint32_t fb = mapa_shared(b_full, 0);
        for (int kb = 0; kb < kblocks; ++kb)
          tma_load_2d_cg2(&tmB, fb, sB + kb * S::kBBytes, kb * BK, nb * BN + (int)rank * S::kBRows);
      }
      for (int i = 0; tile_at(i, mb, nb) && !timed_out; ++i) {
        for (int kb = 0; kb < kblocks; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1)) { timed_out = true; break; }
          uint8_t* da = sA + stage * A_BYTES;
          uint8_t* db = sB + stage * S::kBBytes;
          const int ya = mb * S::kTileM + (int)rank * BM, yb = nb * BN + (int)rank * S::kBRows;
          if constexpr (CG == 2) {
            // both CTAs' halves complete on the leader's barrier, which the
            // leader arms for the bytes of both
            if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * (KEEP_B ? A_BYTES : S::kStageBytes));
            const uint32_t fb = mapa_shared(&full[stage], 0);
            tma_load_2d_cg2(&tmA, fb, da, kb * BK, ya);
            if (!KEEP_B) tma_load_2d_cg2(&tmB, fb, db, kb * BK, yb);
          } else {
            mbar_arrive_expect_tx(&full[stage], S::kStageBytes);
            tma_load_2d(&tmA, &full[stage], da, kb * BK, ya);
            tma_load_2d(&tmB, &full[stage], db, kb * BK, yb);
          }
          if (++stage == NST) { stage = 0; phase ^= 1; }
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      constexpr uint32_t idesc = idesc_i8(S::kTileM, BN);
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      int mb, nb;
      if (KEEP_B && tile_at(0, mb, nb)) timed_out = !mbar_wait(b_full, 0);
      for (int i = 0; tile_at(i, mb, nb) && !timed_out; ++i) {
        if (!mbar_wait(&acc_empty[acc], acc_phase ^ 1)) { timed_out = true; break; }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * BN;
        for (int kb = 0; kb < kblocks; ++kb) {
          if (!mbar_wait(&full[stage], phase)) { timed_out = true; break; }
          tc_fence_after();
          const uint32_t a_addr = smem_u32(sA + stage * A_BYTES);
          const uint32_t b_addr = smem_u32(sB + (KEEP_B ? kb : stage) * S::kBBytes);
#pragma unroll
          for (int k = 0; k < BK / 32; ++k)
            mma_i8<CG>(d_tmem, sdesc_sw128(a_addr + 32 * k, 16, 1024), sdesc_sw128(b_addr + 32 * k, 16, 1024),
                       idesc, (kb | k) != 0 ? 1u : 0u);
          if constexpr (CG == 2) tc_commit_cg2(&empty[stage], 0x3);
          else tc_commit(&empty[stage]);
          if (++stage == NST) { stage = 0; phase ^= 1; }
        }
        if (timed_out) break;
        if constexpr (CG == 2) tc_commit_cg2(&acc_full[acc], 0x3);
        else tc_commit(&acc_full[acc]);
        if (++acc == 2) { acc = 0; acc_phase ^= 1; }
      }
    }
  } else {
    // epilogue warp ew drains rows [32 quarter, 32 quarter + 32) of its CTA,
    // the blocks of its column group
    const int quarter = warp & 3, ew = warp - 2;
    constexpr int NB = E::kBlocks;
    const int grp = ew >> 2;
    uint8_t* stg = sStg + ew * E::kBufs * E::kStg;
    // the output is not read here: its lines leave L2 first (154 -> 152.7 us at
    // 131075 x 2048 x 512 to f16)
    const uint64_t evict_first = policy_evict_first();
    int acc = 0;
    uint32_t acc_phase = 0, chunk = 0;
    // the residual comes by plain loads into a ring of two blocks, ahead of use
    // and across tile boundaries, so that its latency hides behind the drain
    constexpr int RB = EPI == MTGR_EPI_RESID ? 2 : 1;
    static_assert(EPI != MTGR_EPI_RESID || NB % RB == 0, "a block's ring slot is its index mod RB");
    float4 rs[RB][8];
    int li = 0, lc = 0;  // the next block to load
    auto load_next = [&](float4 (&z)[8]) {
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      int mb, nb;
      if (tile_at(li, mb, nb)) {
        const int m = mb * S::kTileM + (int)rank * BM + quarter * 32 + lane;
        const int col = nb * BN + (grp * NB + lc) * 32;
        if (m < M) {
          const float4* p = reinterpret_cast<const float4*>(args.resid + (size_t)m * N + col);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (col + 4 * i < N) z[i] = __ldg(p + i);
        }
      }
      if (++lc == NB) { lc = 0; ++li; }
    };
    if constexpr (EPI == MTGR_EPI_RESID) {
#pragma unroll
      for (int sl = 0; sl < RB; ++sl) load_next(rs[sl]);
    }
    int mb, nb;
    for (int i = 0; tile_at(i, mb, nb); ++i) {
      const int row0 = mb * S::kTileM + (int)rank * BM + quarter * 32;
      const bool live = row0 + lane < M;
      const float sa = live ? load_written(args.sa + row0 + lane) : 0.f;
      const bool ok = __all_sync(0xffffffffu, mbar_wait(&acc_full[acc], acc_phase));
      if (!ok) { timed_out = true; break; }
      tc_fence_after();
      const uint32_t t_row = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + acc * BN;
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          // the accumulator is released on the leader's barrier (its TMEM loads
          // have completed, so the remote arrive needs no ordering)
          if (CG == 1 || rank == 0) mbar_arrive(&acc_empty[acc]);
          else mbar_arrive_cluster_relaxed(mapa_shared(&acc_empty[acc], 0));
        }
      };
#pragma unroll RB
      for (int cc = 0; cc < NB; ++cc) {
        const int blk = grp * NB + cc;
        const int col0 = nb * BN + blk * E::kCols;
        const bool last = cc == NB - 1;
        if (col0 < N) {
          uint8_t* st = stg + (E::kBufs == 2 ? (chunk & 1) * E::kStg : 0);
          // the TMA store that last read this buffer must be done
          if (lane == 0) bulk_wait_group_read<E::kBufs - 1>();
          __syncwarp();
#pragma unroll
          for (int half = 0; half < E::kCols / 32; ++half) {
            const int col = col0 + 32 * half;
            const bool end = last && half == E::kCols / 32 - 1;
            if (half > 0 && col >= N) {  // nothing of this half is stored
              if (end) release();
              break;
            }
            uint32_t r[32];
            tmem_ld32(t_row + blk * E::kCols + 32 * half, r);
            const auto loaded = [&] { if (end) release(); };
            if (col + 32 <= N)
              epilogue_cols<EPI, OUT, true>(args, col, sa, live, r, rs[cc % RB], st, lane, 4 * half, loaded);
            else
              epilogue_cols<EPI, OUT, false>(args, col, sa, live, r, rs[cc % RB], st, lane, 4 * half, loaded);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d_hint(&tmO, st, col0, row0, evict_first);
            bulk_commit_group();
          }
          ++chunk;
        } else if (last) {
          release();
        }
        if constexpr (EPI == MTGR_EPI_RESID) load_next(rs[cc % RB]);
      }
      if (++acc == 2) { acc = 0; acc_phase ^= 1; }
    }
    if (lane == 0) bulk_wait_group<0>();  // stores complete before the CTA retires
  }
  if (timed_out) set_status(args.status, MTGR_ERR_TIMEOUT);
  // a pair retires together: the leader's MMAs read the other CTA's shared
  // memory and the other CTA arrives on the leader's barriers
  tc_fence_before();
  if constexpr (CG == 2) cluster_sync();
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    if constexpr (CG == 2) tmem_dealloc_cg2(tmem_base, S::kTmemCols);
    else tmem_dealloc(tmem_base, S::kTmemCols);
  }
}

constexpr int kMaxDevices = 64;

// Whether pairs keep b in shared memory (k <= kKeepK), on `units` pairs. A pair stays in one
// column of tiles, so units % n_tiles of them have no work; that has to be little. Where
// rows of k bytes are not whole 128-byte lines, loading b again costs most: kept against
// reloaded 100003 x 2048 x 272 to f16 99 / 114 us, x 448 109 / 118, x 496 125 / 143; up to
// ten of 74 pairs idle it stays ahead (100003 x 4096 x 448 236 / 245), at 14 no more (x 3840:
// 236 / 225). With whole lines it gains at k = 512 alone, with two pairs idle (131075 x 2048 x
// 512 140 / 145, x 2560 with four 189 / 186) and four row tiles a pair (10000 x 1024 x 512,
// two of them: 14.4 / 12.7), and not below (131075 x 2048 x 384 146 / 136, x 256 136 / 125).
inline bool keeps_b(int units, int64_t m_tiles, int n_tiles, int K) {
  if (units < n_tiles) return false;
  const int idle = units % n_tiles;
  if (K % BK != 0) return 7 * idle <= units;
  return K == kKeepK && 32 * idle <= units && m_tiles >= 4 * (units / n_tiles);
}

template <int EPI, int OUT, int CG, bool KEEP_B>
int launch_t(const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& to, const Args& args,
             cudaStream_t s, bool dependent) {
  using E = Epi<OUT, CG, KEEP_B>;
  auto kern = gemm_i8_kernel<EPI, OUT, CG, KEEP_B>;
  // per device: blocks (pairs) resident at once; 0 until the first launch there
  static std::atomic<int> resident[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return MTGR_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(E::kThreads);
  cfg.dynamicSmemBytes = E::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CG;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int units = resident[dev].load(std::memory_order_relaxed);
  if (units == 0) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)E::kSmem) != cudaSuccess)
      return MTGR_ERR_CUDA;
    units = device_sm_count();
    if (CG == 2) {  // a GPC with an odd number of SMs leaves one unpaired
      cfg.gridDim = dim3(units);
      int n = 0;
      if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n <= 0) return MTGR_ERR_CUDA;
      units = n;
    }
    resident[dev].store(units, std::memory_order_relaxed);
  }
  const int n_tiles = (args.N + Shape<CG>::kBN - 1) / Shape<CG>::kBN;
  const int64_t m_tiles = ((int64_t)args.M + BM * CG - 1) / (BM * CG), tiles = m_tiles * n_tiles;
  if (KEEP_B && !keeps_b(units, m_tiles, n_tiles, args.K))
    return launch_t<EPI, OUT, CG, false>(ta, tb, to, args, s, dependent);
  if (tiles > 0x3fffffff) return MTGR_ERR_UNSUPPORTED;  // the kernel counts tiles in 32 bits
  cfg.gridDim = dim3((unsigned)(CG * (tiles < units ? tiles : units)));
  cfg.numAttrs = dependent ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kern, ta, tb, to, args) != cudaSuccess) return MTGR_ERR_CUDA;
  return launch_status();
}

template <int CG>
int launch_cg(int M, int N, int K, const int8_t* a, const int8_t* b, int epi, int32_t out_dtype, void* out,
              const Args& args, cudaStream_t s, bool dependent) {
  using S = Shape<CG>;
  CUtensorMap ta, tb, to;
  int rc = make_tmap_2d(&ta, a, CU_TENSOR_MAP_DATA_TYPE_UINT8, (uint64_t)K, (uint64_t)M, (uint64_t)K, BK, BM,
                        CU_TENSOR_MAP_SWIZZLE_128B);
  if (rc != MTGR_OK) return rc;
  rc = make_tmap_2d(&tb, b, CU_TENSOR_MAP_DATA_TYPE_UINT8, (uint64_t)K, (uint64_t)N, (uint64_t)K, BK,
                    S::kBRows, CU_TENSOR_MAP_SWIZZLE_128B);
  if (rc != MTGR_OK) return rc;
  rc = out_dtype == MTGR_F32
           ? make_tmap_2d(&to, out, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, (uint64_t)N, (uint64_t)M,
                          (uint64_t)N * 4, 32, 32, CU_TENSOR_MAP_SWIZZLE_128B)
           : make_tmap_2d(&to, out, CU_TENSOR_MAP_DATA_TYPE_UINT16, (uint64_t)N, (uint64_t)M,
                          (uint64_t)N * 2, 64, 32, CU_TENSOR_MAP_SWIZZLE_128B);
  if (rc != MTGR_OK) return rc;
  // b's tile may stay where k is short and every column of tiles has four pairs or more
  const bool keep = CG == 2 && K <= kKeepK && (N + S::kBN - 1) / S::kBN <= device_sm_count() / 8;
#define MTGR_FORM(E, O) \
  if (epi == E && out_dtype == O)                                                     \
    return keep ? launch_t<E, O, CG, CG == 2>(ta, tb, to, args, s, dependent)          \
                : launch_t<E, O, CG, false>(ta, tb, to, args, s, dependent)
  MTGR_FORM(MTGR_EPI_NONE, MTGR_F16);
  MTGR_FORM(MTGR_EPI_NONE, MTGR_BF16);
  MTGR_FORM(MTGR_EPI_NONE, MTGR_F32);
  MTGR_FORM(MTGR_EPI_SILU, MTGR_F16);
  MTGR_FORM(MTGR_EPI_SILU, MTGR_BF16);
  MTGR_FORM(MTGR_EPI_SILU, MTGR_F32);
  MTGR_FORM(MTGR_EPI_RESID, MTGR_F32);
#undef MTGR_FORM
  return MTGR_ERR_UNSUPPORTED;
}

// ------------------------------------------------ few tiles and a long k --
// A cluster of `splits` CTAs shares one 128 x 64 tile: each multiplies its run of
// k-blocks, leaves its int32 sums in its shared memory, and after a cluster barrier
// finishes its share of the rows from all of theirs. Sums of integers: the
// same bits as in one run over k.
constexpr int kSplitK = 16;  // fewest k-blocks
constexpr int kSplitThreads = 192, kSplitStages = 6;
constexpr int kSplitRows = (BM / 2 * 8 + kSplitThreads - 1) / kSplitThreads;  // rows a thread finishes, at two splits
constexpr size_t kSplitSmem = 1024 + (size_t)kSplitStages * Shape<1>::kStageBytes + 256;

// 16-byte chunk c of row r of a tile of 64 int32 columns: chunks turned by the row, so that
// eight rows' same chunk falls in different banks
__device__ __forceinline__ uint32_t part_off(int r, int c) { return (uint32_t)(r * 256 + ((c ^ (r & 7)) << 4)); }

__device__ __forceinline__ int4 ld_peer(uint32_t addr) {
  int4 v;
  asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

template <int OUT>
__global__ void __launch_bounds__(kSplitThreads, 1)
    gemm_i8_split_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, Args args,
                         int splits, int epi, void* out) {
  using S = Shape<1>;
  constexpr int NST = kSplitStages, BN = S::kBN;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + NST * A_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(sB + NST * S::kBBytes);
  uint64_t* empty = full + NST;
  uint64_t* done = full + 2 * NST;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(full + 2 * NST + 1);

  const int warp = warp_id(), lane = lane_id();
  const int M = args.M, N = args.N;
  const int n_tiles = (N + BN - 1) / BN, tile = (int)blockIdx.x / splits;
  const int mb = tile / n_tiles, nb = tile - mb * n_tiles;
  const int rank = (int)cluster_ctarank();
  const int kblocks = (args.K + BK - 1) / BK;  // kSplitK at least
  const int k0 = rank * kblocks / splits, k1 = (rank + 1) * kblocks / splits;

  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    for (int s = 0; s < NST; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, BN);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  bool timed_out = false;
  dependent_wait();  // a's bytes and scales may be another kernel's of the same call

  // what finishing takes beside the sums, on its way while k is added up: the scales and the
  // bias of a thread's eight columns (the same in each of its rows), its rows' scales
  const int rows = BM / splits, n = nb * BN + 8 * (int)(threadIdx.x & 7);
  float sb[8], bias[8], sa[kSplitRows];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    sb[e] = n < N ? __ldg(args.sb + n + e) : 0.f;  // N % 8 == 0
    bias[e] = n < N && args.bias != nullptr ? __ldg(args.bias + n + e) : 0.f;
  }
#pragma unroll
  for (int i = 0; i < kSplitRows; ++i) {
    const int r = i * (kSplitThreads / 8) + (int)(threadIdx.x >> 3), m = mb * BM + rank * rows + r;
    sa[i] = r < rows && m < M ? load_written(args.sa + m) : 0.f;
  }

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      for (int kb = k0; kb < k1; ++kb) {
        if (!mbar_wait(&empty[stage], phase ^ 1)) { timed_out = true; break; }
        mbar_arrive_expect_tx(&full[stage], S::kStageBytes);
        tma_load_2d(&tmA, &full[stage], sA + stage * A_BYTES, kb * BK, mb * BM);
        tma_load_2d(&tmB, &full[stage], sB + stage * S::kBBytes, kb * BK, nb * BN);
        if (++stage == NST) { stage = 0; phase ^= 1; }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_i8(BM, BN);
      int stage = 0;
      uint32_t phase = 0;
      for (int kb = k0; kb < k1; ++kb) {
        if (!mbar_wait(&full[stage], phase)) { timed_out = true; break; }
        tc_fence_after();
        const uint32_t a_addr = smem_u32(sA + stage * A_BYTES), b_addr = smem_u32(sB + stage * S::kBBytes);
#pragma unroll
        for (int k = 0; k < BK / 32; ++k)
          mma_i8<1>(tmem_base, sdesc_sw128(a_addr + 32 * k, 16, 1024), sdesc_sw128(b_addr + 32 * k, 16, 1024), idesc,
                    kb > k0 || k > 0 ? 1u : 0u);
        tc_commit(&empty[stage]);
        if (++stage == NST) { stage = 0; phase ^= 1; }
      }
      if (!timed_out) tc_commit(done);
    }
  } else {
    // all multiplications done, so all loads landed: the stages of a take the sums
    if (__all_sync(0xffffffffu, mbar_wait(done, 0))) {
      tc_fence_after();
      const int r = 32 * (warp & 3) + lane;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t v[32];
        tmem_ld32(tmem_base + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + 32 * half, v);
        tmem_ld_wait();
        reg_fence(v);
#pragma unroll
        for (int c = 0; c < 8; ++c)
          *reinterpret_cast<uint4*>(sA + part_off(r, 8 * half + c)) =
              make_uint4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
      }
    } else {
      timed_out = true;
    }
  }
  tc_fence_before();
  cluster_sync();
  // this CTA's rows of the tile, eight columns a thread
  const int c = threadIdx.x & 7;
#pragma unroll
  for (int i = 0; i < kSplitRows; ++i) {
    const int ri = i * (kSplitThreads / 8) + (int)(threadIdx.x >> 3), r = rank * rows + ri, m = mb * BM + r;
    if (ri >= rows || m >= M || n >= N) continue;
    int4 lo = make_int4(0, 0, 0, 0), hi = lo;
#pragma unroll 4
    for (int p = 0; p < splits; ++p) {
      const uint32_t from = mapa_shared(sA, (uint32_t)p);
      const int4 x = ld_peer(from + part_off(r, 2 * c)), y = ld_peer(from + part_off(r, 2 * c + 1));
      lo.x += x.x; lo.y += x.y; lo.z += x.z; lo.w += x.w;
      hi.x += y.x; hi.y += y.y; hi.z += y.z; hi.w += y.w;
    }
    const int s[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      // rounded step by step, as in the other forms
      v[e] = __fmul_rn(__int2float_rn(s[e]), __fmul_rn(sa[i], sb[e]));
      if (args.bias != nullptr) v[e] = __fadd_rn(v[e], bias[e]);
      if (epi == MTGR_EPI_SILU) v[e] = __fdividef(v[e], 1.0f + __expf(-v[e]));
      if (epi == MTGR_EPI_RESID) v[e] = __fadd_rn(v[e], __ldg(args.resid + (size_t)m * N + n + e));
      if (n < args.q_cols) v[e] = __fmul_rn(v[e], 0.5f);  // q_cols % 32 == 0
    }
    if (OUT == MTGR_F32) {
      store8(static_cast<float*>(out) + (size_t)m * N + n, v);
    } else if (OUT == MTGR_BF16) {
      store8(static_cast<__nv_bfloat16*>(out) + (size_t)m * N + n, v);
    } else {
      float mx = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(v[e]));
      if (mx > 65504.f) set_status(args.status, MTGR_ERR_RANGE);
      *reinterpret_cast<uint4*>(static_cast<__half*>(out) + (size_t)m * N + n) =
          make_uint4(cvt_f16x2(v[0], v[1]), cvt_f16x2(v[2], v[3]), cvt_f16x2(v[4], v[5]), cvt_f16x2(v[6], v[7]));
    }
  }
  if (timed_out) set_status(args.status, MTGR_ERR_TIMEOUT);
  cluster_sync();  // no CTA ends while another reads its sums
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, BN);
  }
}

template <int OUT>
int launch_split_t(const CUtensorMap& ta, const CUtensorMap& tb, const Args& args, int tiles, int splits, int epi,
                   void* out, cudaStream_t s, bool dependent) {
  auto kern = gemm_i8_split_kernel<OUT>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSplitSmem) != cudaSuccess)
    return MTGR_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * splits));
  cfg.blockDim = dim3(kSplitThreads);
  cfg.dynamicSmemBytes = kSplitSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)splits;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = dependent ? 2 : 1;
  cudaLaunchKernelEx(&cfg, kern, ta, tb, args, splits, epi, out);
  return launch_status();
}

int launch_split(int M, int N, int K, const int8_t* a, const int8_t* b, int epi, int32_t out_dtype, void* out,
                 const Args& args, int splits, cudaStream_t s, bool dependent) {
  CUtensorMap ta, tb;
  int rc = make_tmap_2d(&ta, a, CU_TENSOR_MAP_DATA_TYPE_UINT8, (uint64_t)K, (uint64_t)M, (uint64_t)K, BK, BM,
                        CU_TENSOR_MAP_SWIZZLE_128B);
  if (rc != MTGR_OK) return rc;
  rc = make_tmap_2d(&tb, b, CU_TENSOR_MAP_DATA_TYPE_UINT8, (uint64_t)K, (uint64_t)N, (uint64_t)K, BK, Shape<1>::kBRows,
                    CU_TENSOR_MAP_SWIZZLE_128B);
  if (rc != MTGR_OK) return rc;
  const int tiles = ((M + BM - 1) / BM) * ((N + Shape<1>::kBN - 1) / Shape<1>::kBN);
  if (out_dtype == MTGR_F32) return launch_split_t<MTGR_F32>(ta, tb, args, tiles, splits, epi, out, s, dependent);
  if (out_dtype == MTGR_BF16) return launch_split_t<MTGR_BF16>(ta, tb, args, tiles, splits, epi, out, s, dependent);
  return launch_split_t<MTGR_F16>(ta, tb, args, tiles, splits, epi, out, s, dependent);
}

}  // namespace

// K % 16 == 0, N % 8 == 0, 16-byte aligned operands.
int launch_gemm_i8(int M, int N, int K, const int8_t* a, const float* sa, const int8_t* b, const float* sb,
                   const float* bias, int epi, const float* resid, int q_cols, int32_t out_dtype, void* out,
                   int32_t* status, cudaStream_t s, bool dependent) {
  if (M == 0 || N == 0) return MTGR_OK;
  const Args args{M, N, K, sa, sb, bias, resid, q_cols, status};
  // Small tiles spread the work while they need at most two rounds of the SMs: 1000 x
  // 2048 x 512 takes 6.5 us in 256 of them, 7.9 in pair tiles; 1000 x 4096 x 1024, 512
  // of them, 14.1 against 8.8.
  const int64_t small_tiles = (((int64_t)M + 127) / 128) * ((N + 63) / 64);
  if (small_tiles > 2 * device_sm_count()) return launch_cg<2>(M, N, K, a, b, epi, out_dtype, out, args, s, dependent);
  // Few tiles and a long k: a cluster of two or four per tile, if the SMs hold them and k
  // has kSplitK blocks. 100 x 1024 x 4096 takes 7.9 us in fours, 12.6 unsplit; 500 x 1024 x
  // 4096, in twos, 10.3 against 12.9; 128 x 512 x 2048 6.8 against 8.1; but 300 x 1024 x
  // 1024 6.7 against 6.0: the cluster and the exchange cost 1.2 us. Eights take 13.6 for
  // the first (a cluster stays in its GPC, and sixteen of eight do not fit at once).
  int splits = 4;
  while (splits > 1 && small_tiles * splits > device_sm_count()) splits /= 2;
  if ((K + BK - 1) / BK < kSplitK) splits = 1;
  if (splits > 1) return launch_split(M, N, K, a, b, epi, out_dtype, out, args, splits, s, dependent);
  return launch_cg<1>(M, N, K, a, b, epi, out_dtype, out, args, s, dependent);
}

}  // namespace mtgr
