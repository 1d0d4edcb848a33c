// The int8 product for few rows (a chunk of candidates, a single token), in one
// kernel from float rows to the output: latency counts here, not bandwidth.
//
//   out[m][n] = epi(sa[m] sb[n] sum_k a[m][k] b[n][k] + bias[n]),  M <= 16
//
// A block takes 16 output channels. Its warps first ask for their share of the
// weights (each warp an eighth of k: 16 bytes a lane and load), then quantise the
// rows into shared memory (every block does it anew: the rows are a few KB out of
// L2, a second kernel would cost more than it saves), then multiply with
// mma.sync m16n8k32 on signed bytes. The k order within an instruction does not
// matter as long as a and b share it, so a lane's 16 consecutive bytes serve two
// instructions. The warps' exact int32 sums meet in shared memory.
// In a graph, bf16 rows, against the quantiser and 128 x 64 tcgen05 tiles: 8 x 2048 x
// 512 3.5 us (5.4 there), 8 x 1024 x 4096 8.7 (14.2), 16 x 4096 x 1024 5.4 (7.2). With
// more rows, or with more blocks than two an SM, quantising in every block costs
// more than it saves: 32 x 2048 x 512 took 6.4 (5.4), 16 x 8192 x 512 7.7 (6.2).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "ops.h"
#include "rowvec.cuh"

namespace mtgr {

namespace {

constexpr int kWarps = 8;
constexpr int kRows = 16;      // rows of an instruction
constexpr int kCols = 16;      // output channels a block
constexpr int kAheadK = 4;     // 64-byte k groups a warp has in flight per channel tile

struct FewArgs {
  int M, N, K;
  const void* x;  // rows: int8 (with sa) or float
  int64_t ld_x;
  const float* sa;
  const int8_t* b;
  const float* sb;
  const float* bias;
  const float* resid;
  void* out;
  int q_cols;
  int32_t* status;
};

__device__ __forceinline__ void mma_s8(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Row r of x to bytes in shared memory (K % 16 == 0 of them, then zeros to the next
// 64), by one warp; returns its scale. Rows of another type are read twice, the
// second time from L1.
template <typename TX>
__device__ __forceinline__ float take_row(const FewArgs& a, int r, uint8_t* to, int lane) {
  const int nv = a.K >> 3;
  float s;
  if constexpr (sizeof(TX) == 1) {
    const uint2* from = reinterpret_cast<const uint2*>(static_cast<const int8_t*>(a.x) + (int64_t)r * a.ld_x);
    for (int vi = lane; vi < nv; vi += 32) *reinterpret_cast<uint2*>(to + 8 * vi) = from[vi];
    s = a.sa[r];
  } else {
    const TX* from = static_cast<const TX*>(a.x) + (int64_t)r * a.ld_x;
    float mx = 0.f;
#pragma unroll 4
    for (int vi = lane; vi < nv; vi += 32) {
      Vec8<TX> w;
      w.load(from + 8 * vi);
      mx = max_nan(mx, max_abs8(w));
    }
    const RowScale rs = row_scale(__reduce_max_sync(0xffffffffu, __float_as_uint(mx)));
#pragma unroll 4
    for (int vi = lane; vi < nv; vi += 32) {
      Vec8<TX> w;
      w.load(from + 8 * vi);
      f2 v[4];
      w.pairs(v);
      *reinterpret_cast<uint2*>(to + 8 * vi) = quant8(v, rs);
    }
    s = rs.s;
  }
  for (int vi = nv + lane; vi < ((a.K + 63) >> 6) * 8; vi += 32) *reinterpret_cast<uint2*>(to + 8 * vi) = make_uint2(0u, 0u);
  return s;
}

template <typename TX>
__global__ void __launch_bounds__(32 * kWarps) gemm_i8_few_kernel(FewArgs a, int epi, int out_dtype) {
  extern __shared__ __align__(16) uint8_t rows[];  // [16][stride], then the warps' sums
  __shared__ float row_s[kRows];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, q = lane & 3;  // the lane's row (channel) and its 16 bytes of a k group
  const int groups = (a.K + 63) >> 6;
  const int stride = groups * 64 + 64;  // rows 64 bytes off, so that a row pair's reads miss each other's banks
  const int n0 = blockIdx.x * kCols;
  const int per = (groups + kWarps - 1) / kWarps;
  const int g0 = warp * per, g1 = min(groups, g0 + per);
  // the first weights, under way while the rows are quantised
  uint4 w[2][kAheadK];
  auto fetch = [&](int kg, uint4 (&d)[2][kAheadK], int slot) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int n = n0 + 8 * t + g, k = 64 * kg + 16 * q;
      d[t][slot] = make_uint4(0u, 0u, 0u, 0u);
      if (kg < g1 && n < a.N && k < a.K)
        d[t][slot] = __ldg(reinterpret_cast<const uint4*>(a.b + (int64_t)n * a.K + k));
    }
  };
#pragma unroll
  for (int i = 0; i < kAheadK; ++i) fetch(g0 + i, w, i);
  for (int r = warp; r < kRows; r += kWarps) {
    if (r < a.M) {
      const float s = take_row<TX>(a, r, rows + r * stride, lane);
      if (lane == 0) row_s[r] = s;
    } else {
      for (int i = lane; i < groups * 8; i += 32) *reinterpret_cast<uint2*>(rows + r * stride + 8 * i) = make_uint2(0u, 0u);
    }
  }
  __syncthreads();
  int c[2][4] = {};
  for (int kg = g0; kg < g1; kg += kAheadK) {
#pragma unroll
    for (int i = 0; i < kAheadK; ++i) {
      if (kg + i < g1) {
        const uint8_t* p = rows + g * stride + 64 * (kg + i) + 16 * q;
        const uint4 x = *reinterpret_cast<const uint4*>(p), y = *reinterpret_cast<const uint4*>(p + 8 * stride);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          mma_s8(c[t], x.x, y.x, x.y, y.y, w[t][i].x, w[t][i].y);
          mma_s8(c[t], x.z, y.z, x.w, y.w, w[t][i].z, w[t][i].w);
        }
      }
      fetch(kg + kAheadK + i, w, i);
    }
  }
  // the warps' sums: [warp][row][channel]
  __syncthreads();  // the rows are done with: their memory takes the sums
  int* part = reinterpret_cast<int*>(rows);
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    int* p = part + (warp * kRows + g) * kCols + 8 * t + 2 * q;
    p[0] = c[t][0];
    p[1] = c[t][1];
    p[8 * kCols] = c[t][2];
    p[8 * kCols + 1] = c[t][3];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kRows * kCols; i += 32 * kWarps) {
    const int m = i / kCols, n = n0 + i % kCols;
    if (m >= a.M || n >= a.N) continue;
    int s = 0;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) s += part[k * kRows * kCols + i];
    // rounded step by step, as in the other forms: a row's bits do not depend on how many
    // rows share the call
    float v = __fmul_rn(__int2float_rn(s), __fmul_rn(row_s[m], a.sb[n]));
    if (a.bias != nullptr) v = __fadd_rn(v, a.bias[n]);
    if (epi == MTGR_EPI_SILU) v = __fdividef(v, 1.0f + __expf(-v));
    const int64_t at = (int64_t)m * a.N + n;
    if (epi == MTGR_EPI_RESID) v = __fadd_rn(v, a.resid[at]);
    if (n < a.q_cols) v = __fmul_rn(v, 0.5f);
    if (out_dtype == MTGR_F32) {
      static_cast<float*>(a.out)[at] = v;
    } else if (out_dtype == MTGR_BF16) {
      static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(v);
    } else {
      // as the tiled forms: beyond f16 saturates and is reported
      if (fabsf(v) > 65504.f) set_status(a.status, MTGR_ERR_RANGE);
      const float lim = v > 65504.f ? 65504.f : (v < -65504.f ? -65504.f : v);
      static_cast<__half*>(a.out)[at] = __float2half_rn(lim);
    }
  }
}

constexpr int kMaxRowsBytes = 100 * 1024;

int smem_bytes(int K) {
  const int rows = kRows * (((K + 63) / 64) * 64 + 64), sums = kWarps * kRows * kCols * 4;
  return rows > sums ? rows : sums;
}

template <typename TX>
int launch_t(const FewArgs& a, int epi, int32_t out_dtype, cudaStream_t s) {
  const int bytes = smem_bytes(a.K);
  auto kern = gemm_i8_few_kernel<TX>;
  // always the largest: a limit set to this call's bytes could fall below what another
  // thread, between its own setting and its launch, is about to ask for
  if (bytes > 40 * 1024 &&
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxRowsBytes) != cudaSuccess)
    return MTGR_ERR_CUDA;
  kern<<<(a.N + kCols - 1) / kCols, 32 * kWarps, bytes, s>>>(a, epi, out_dtype);
  return launch_status();
}

}  // namespace

// Few rows and channels: one instruction's rows, at most two blocks an SM, and a
// block's bytes of the rows fit its shared memory.
bool gemm_i8_is_few(int32_t M, int32_t N, int32_t K) {
  return M <= kRows && N <= kCols * 2 * device_sm_count() && K <= 8192 && smem_bytes(K) <= kMaxRowsBytes;
}

// x_dtype MTGR_I8: x are bytes with scales sa; else float rows, quantised here.
int launch_gemm_i8_few(int M, int N, int K, int32_t x_dtype, const void* x, int64_t ld_x, const float* sa,
                       const int8_t* b, const float* sb, const float* bias, int epi, const float* resid, int q_cols,
                       int32_t out_dtype, void* out, int32_t* status, cudaStream_t s) {
  if (M == 0 || N == 0) return MTGR_OK;
  const FewArgs a{M, N, K, x, ld_x, sa, b, sb, bias, resid, out, q_cols, status};
  switch (x_dtype) {
    case MTGR_I8: return launch_t<int8_t>(a, epi, out_dtype, s);
    case MTGR_F32: return launch_t<float>(a, epi, out_dtype, s);
    case MTGR_BF16: return launch_t<__nv_bfloat16>(a, epi, out_dtype, s);
    case MTGR_F16: return launch_t<__half>(a, epi, out_dtype, s);
    default: return MTGR_ERR_UNSUPPORTED;
  }
}

}  // namespace mtgr
