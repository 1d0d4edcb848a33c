// Arguments and launchers of the block-boundary, int8 and gradient-clipping
// operators (boundary.cu, quant.cu, gemm_i8.cu, grad_clip.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/mtgr.h"

namespace mtgr {

// A kernel that follows another of the same call may be launched while that one
// still runs: its blocks take their places and wait (dependent_wait, before their
// first access to memory) until the first kernel has ended and its writes are
// seen. The first one allows it as soon as all of its blocks run.
__device__ __forceinline__ void dependents_may_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void dependent_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Reads what was written while this kernel ran, by the kernel before it or by another block: behind
// the wait for it in the program, where __ldg (memory that never changes) may go ahead of it.
__device__ __forceinline__ float load_written(const float* p) {
  float v;
  asm volatile("ld.relaxed.gpu.global.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ double load_written(const double* p) {
  double v;
  asm volatile("ld.relaxed.gpu.global.f64 %0, [%1];" : "=d"(v) : "l"(p) : "memory");
  return v;
}

template <typename... P, typename... A>
inline int launch_dependent(void (*kern)(P...), unsigned grid, unsigned block, size_t smem, cudaStream_t s,
                            A&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, P(args)...) != cudaSuccess) return MTGR_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? MTGR_OK : MTGR_ERR_CUDA;
}

constexpr int kMaxGroups = 32;  // the backward keeps the groups a team saw in 32 bits

struct BoundaryFwdArgs {
  int32_t T, d, G, gate;
  float eps;
  const int8_t* gid;
  const void *o, *u, *x;
  int64_t ld_o, ld_u;
  const float *post_gamma, *post_beta, *scale, *pre_gamma, *pre_beta;
  void *h, *y;
  int32_t y_dtype;
  float* y_scale;
};

struct BoundaryBwdArgs {
  int32_t T, d, G, gate, o_dtype, dy_dtype;
  float eps;
  const int8_t* gid;
  const void *o, *u, *x, *dh, *dy;
  int64_t ld_o, ld_u, ld_do, ld_du;
  const float *post_gamma, *post_beta, *scale, *pre_gamma, *pre_beta;
  void *d_o, *du, *dx;
  float *g_post_gamma, *g_post_beta, *g_scale, *g_pre_gamma, *g_pre_beta;
  int32_t* status;
  // filled by the launcher
  int32_t teams, rows_per_team;
  uint32_t* seen;
  float* part;
};

int launch_boundary_fwd(const BoundaryFwdArgs& a, int32_t o_dtype, int32_t x_dtype, cudaStream_t s);
size_t boundary_bwd_ws_bytes(int32_t T, int32_t d, int32_t G);
int launch_boundary_bwd(BoundaryBwdArgs a, int32_t x_dtype, void* ws, cudaStream_t s);

int launch_quantize_rows(int32_t M, int32_t K, int32_t x_dtype, const void* x, int64_t ld_x, int8_t* q,
                         float* scale, cudaStream_t s);

// out[m][n] = epi(sa[m] sb[n] sum_k a[m][k] b[n][k] + bias[n])
int launch_gemm_i8(int M, int N, int K, const int8_t* a, const float* sa, const int8_t* b,
                   const float* sb, const float* bias, int epi, const float* resid, int q_cols,
                   int32_t out_dtype, void* out, int32_t* status, cudaStream_t s, bool dependent = false);

// the same in one kernel from float rows or bytes (MTGR_I8, with sa), for few rows
bool gemm_i8_is_few(int32_t M, int32_t N, int32_t K);
int launch_gemm_i8_few(int M, int N, int K, int32_t x_dtype, const void* x, int64_t ld_x, const float* sa,
                       const int8_t* b, const float* sb, const float* bias, int epi, const float* resid, int q_cols,
                       int32_t out_dtype, void* out, int32_t* status, cudaStream_t s);

size_t grad_clip_ws_bytes(const mtgr_grad_tensor* g, int32_t n);
int grad_clip_launches(const mtgr_grad_tensor* g, int32_t n);
int launch_grad_clip(const mtgr_grad_tensor* g, int32_t n, float max_norm, float inv_scale, float* norm,
                     void* ws, int32_t* status, cudaStream_t s);

}  // namespace mtgr
