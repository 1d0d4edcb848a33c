// Rows to signed bytes with a scale each, for the int8 product:
//   s_m = max(max_k |x_mk|, 2^-100) * (1 / 127),  q_mk = x_mk / s_m to the nearest integer, ties to even
// (rowvec.cuh has the rounding, which is exact). A row is read once and stays in
// registers between its maximum and its bytes; bound by HBM: sizeof(x) + 1
// bytes an element.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "ops.h"
#include "rowvec.cuh"

namespace mtgr {

namespace {

// One row per warp (THREADS = 32, eight rows a block) or per block of THREADS;
// VPL vectors of eight per thread.
template <typename T, int THREADS, int VPL>
__global__ void __launch_bounds__(THREADS == 32 ? 256 : THREADS)
    quantize_rows_kernel(int32_t M, int32_t K, const T* x, int64_t ld_x, int8_t* q, float* scale) {
  constexpr bool BLOCK = THREADS != 32;
  __shared__ uint32_t part[BLOCK ? 32 : 1];
  dependents_may_launch();
  const int tl = threadIdx.x % THREADS;
  const int64_t m = BLOCK ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (m >= M) return;
  const int nv = K >> 3;
  Vec8<T> r[VPL];
#pragma unroll
  for (int k = 0; k < VPL; ++k) {
    const int vi = tl + THREADS * k;
    if (vi < nv) r[k].load(x + m * ld_x + 8 * vi);
  }
  float mx = 0.f;
#pragma unroll
  for (int k = 0; k < VPL; ++k)
    if (tl + THREADS * k < nv) mx = max_nan(mx, max_abs8(r[k]));
  const RowScale rs = row_scale(team_max_bits<BLOCK>(__float_as_uint(mx), part));
  if (tl == 0) scale[m] = rs.s;
#pragma unroll
  for (int k = 0; k < VPL; ++k) {
    const int vi = tl + THREADS * k;
    if (vi < nv) {
      f2 v[4];
      r[k].pairs(v);
      *reinterpret_cast<uint2*>(q + m * K + 8 * vi) = quant8(v, rs);
    }
  }
}

template <typename T>
int launch_t(int32_t M, int32_t K, const void* xv, int64_t ld_x, int8_t* q, float* scale, cudaStream_t s) {
  const T* x = static_cast<const T*>(xv);
  const unsigned warps = (unsigned)(((int64_t)M + 7) / 8);
  if (K <= 256) quantize_rows_kernel<T, 32, 1><<<warps, 256, 0, s>>>(M, K, x, ld_x, q, scale);
  else if (K <= 512) quantize_rows_kernel<T, 32, 2><<<warps, 256, 0, s>>>(M, K, x, ld_x, q, scale);
  else if (K <= 1024) quantize_rows_kernel<T, 32, 4><<<warps, 256, 0, s>>>(M, K, x, ld_x, q, scale);
  else if (K <= 2048) quantize_rows_kernel<T, 32, 8><<<warps, 256, 0, s>>>(M, K, x, ld_x, q, scale);
  else if (K <= 4096) quantize_rows_kernel<T, 64, 8><<<M, 64, 0, s>>>(M, K, x, ld_x, q, scale);
  else if (K <= 8192) quantize_rows_kernel<T, 128, 8><<<M, 128, 0, s>>>(M, K, x, ld_x, q, scale);
  else quantize_rows_kernel<T, 512, 8><<<M, 512, 0, s>>>(M, K, x, ld_x, q, scale);
  return launch_status();
}

}  // namespace

// K % 8 == 0, K <= 32768
int launch_quantize_rows(int32_t M, int32_t K, int32_t x_dtype, const void* x, int64_t ld_x, int8_t* q,
                         float* scale, cudaStream_t s) {
  if (M == 0) return MTGR_OK;
  if (x_dtype == MTGR_F32) return launch_t<float>(M, K, x, ld_x, q, scale, s);
  if (x_dtype == MTGR_BF16) return launch_t<__nv_bfloat16>(M, K, x, ld_x, q, scale, s);
  if (x_dtype == MTGR_F16) return launch_t<__half>(M, K, x, ld_x, q, scale, s);
  return MTGR_ERR_UNSUPPORTED;
}

}  // namespace mtgr
