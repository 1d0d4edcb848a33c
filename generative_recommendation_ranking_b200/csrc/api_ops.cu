// extern "C" entry points of the block-boundary, int8 and gradient-clipping
// operators: argument validation and launches.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "common.cuh"
#include "ops.h"
#include "timer.h"

using namespace mtgr;

namespace {

constexpr int32_t kMaxRowD = 8192;         // as for mtgr_group_layernorm
constexpr int32_t kMaxQuantK = 32768;      // a row stays in one block's registers
constexpr int32_t kMaxI8K = 131072;        // exclusive: 2^14 K < 2^31 for any bytes
constexpr int32_t kMaxI8Rows = 1 << 30;    // row and column indices of whole tiles stay in 32 bits
constexpr int64_t kMaxGradElems = 1ll << 38;

inline cudaStream_t as_stream(mtgr_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// rows of ld elements: at least d of them, 16-byte aligned
inline bool ld_ok(int64_t ld, int32_t d) { return ld >= d && ld % 8 == 0; }

int boundary_check(const mtgr_boundary_params* p, int32_t T, int32_t o_dtype, int32_t x_dtype) {
  if (p == nullptr || T < 0 || p->d <= 0 || p->d % 8 != 0 || p->d > kMaxRowD || p->G <= 0 ||
      !(p->eps >= 0.0f))
    return MTGR_ERR_INVALID_ARG;
  if (p->gate != MTGR_GATE_NONE && p->gate != MTGR_GATE_LINEAR && p->gate != MTGR_GATE_SILU)
    return MTGR_ERR_INVALID_ARG;
  if ((p->post_gamma == nullptr) != (p->post_beta == nullptr) ||
      (p->pre_gamma == nullptr) != (p->pre_beta == nullptr))
    return MTGR_ERR_INVALID_ARG;
  if (!aligned16(p->post_gamma) || !aligned16(p->post_beta) || !aligned16(p->scale) ||
      !aligned16(p->pre_gamma) || !aligned16(p->pre_beta))
    return MTGR_ERR_INVALID_ARG;
  if (p->G > kMaxGroups) return MTGR_ERR_UNSUPPORTED;
  if (o_dtype != MTGR_F32 && o_dtype != MTGR_BF16 && o_dtype != MTGR_F16) return MTGR_ERR_UNSUPPORTED;
  if (x_dtype != MTGR_F32 && x_dtype != MTGR_BF16) return MTGR_ERR_UNSUPPORTED;
  return MTGR_OK;
}

// An output that is an operand of its own product: blocks would write what others still read.
bool is_operand(const void* out, const void* a, const void* b) { return out != nullptr && (out == a || out == b); }

// Arguments of the int8 product that do not depend on how a is given.
int gemm_i8_check(int32_t M, int32_t N, int32_t K, const void* b, const float* sb, const float* bias,
                  int32_t epi, const float* resid, int32_t q_cols, int32_t out_dtype, const void* out) {
  if (M < 0 || N < 0 || K <= 0 || q_cols < 0 || q_cols % 32 != 0) return MTGR_ERR_INVALID_ARG;
  if (epi != MTGR_EPI_NONE && epi != MTGR_EPI_SILU && epi != MTGR_EPI_RESID) return MTGR_ERR_INVALID_ARG;
  if (epi == MTGR_EPI_RESID && (out_dtype != MTGR_F32 || (out != nullptr && resid == out))) return MTGR_ERR_INVALID_ARG;
  if (out_dtype != MTGR_F32 && out_dtype != MTGR_BF16 && out_dtype != MTGR_F16) return MTGR_ERR_UNSUPPORTED;
  if (K % 16 != 0 || N % 8 != 0 || K >= kMaxI8K || M > kMaxI8Rows || N > kMaxI8Rows) return MTGR_ERR_UNSUPPORTED;
  if (M > 0 && N > 0 &&
      (b == nullptr || sb == nullptr || out == nullptr || (epi == MTGR_EPI_RESID && resid == nullptr)))
    return MTGR_ERR_INVALID_ARG;
  if (!aligned16(b) || !aligned16(sb) || !aligned16(bias) || !aligned16(resid) || !aligned16(out))
    return MTGR_ERR_INVALID_ARG;
  return MTGR_OK;
}

int quant_check(int32_t M, int32_t K, int32_t x_dtype, const void* x, int64_t ld_x) {
  if (M < 0 || K <= 0 || !ld_ok(ld_x, K)) return MTGR_ERR_INVALID_ARG;
  if (K % 8 != 0 || K > kMaxQuantK) return MTGR_ERR_UNSUPPORTED;
  if (x_dtype != MTGR_F32 && x_dtype != MTGR_BF16 && x_dtype != MTGR_F16) return MTGR_ERR_UNSUPPORTED;
  if ((M > 0 && x == nullptr) || !aligned16(x)) return MTGR_ERR_INVALID_ARG;
  return MTGR_OK;
}

int grads_check(const mtgr_grad_tensor* g, int32_t n) {
  if (n < 0 || (n > 0 && g == nullptr)) return MTGR_ERR_INVALID_ARG;
  int32_t first = -1;  // the first tensor that is not empty
  for (int32_t i = 0; i < n; ++i) {
    if (g[i].n < 0 || g[i].n > kMaxGradElems || (g[i].n > 0 && g[i].g == nullptr)) return MTGR_ERR_INVALID_ARG;
    const int e = dtype_size(g[i].dtype), eo = dtype_size(g[i].out_dtype);
    if (e == 0 || eo == 0) return MTGR_ERR_UNSUPPORTED;
    if (g[i].out_dtype != g[i].dtype && g[i].out_dtype != MTGR_F32) return MTGR_ERR_UNSUPPORTED;
    if (reinterpret_cast<uintptr_t>(g[i].g) % e != 0 || reinterpret_cast<uintptr_t>(g[i].out) % eo != 0)
      return MTGR_ERR_INVALID_ARG;
    // in place only in the same type; outputs for all tensors or for none
    if (g[i].out == g[i].g && g[i].out != nullptr && g[i].out_dtype != g[i].dtype) return MTGR_ERR_INVALID_ARG;
    if (g[i].n == 0) continue;
    if (first < 0) first = i;
    if ((g[i].out == nullptr) != (g[first].out == nullptr)) return MTGR_ERR_INVALID_ARG;
  }
  return MTGR_OK;
}

}  // namespace

extern "C" {

MTGR_API int mtgr_boundary_fwd(const mtgr_boundary_params* p, int32_t T, const int8_t* d_group_id,
                               int32_t o_dtype, const void* d_o, int64_t ld_o, const void* d_u, int64_t ld_u,
                               int32_t x_dtype, const void* d_x, void* d_h, int32_t y_dtype, void* d_y,
                               float* d_y_scale, mtgr_stream_t stream) {
  const int rc = boundary_check(p, T, o_dtype, x_dtype);
  if (rc != MTGR_OK) return rc;
  const bool gate = p->gate != MTGR_GATE_NONE, pre = p->pre_gamma != nullptr;
  if (pre && y_dtype != MTGR_F32 && y_dtype != MTGR_BF16 && y_dtype != MTGR_I8) return MTGR_ERR_UNSUPPORTED;
  if (!ld_ok(ld_o, p->d) || (gate && !ld_ok(ld_u, p->d))) return MTGR_ERR_INVALID_ARG;
  if (T > 0 && (d_group_id == nullptr || d_o == nullptr || (gate && d_u == nullptr) || d_x == nullptr ||
                d_h == nullptr || (pre && (d_y == nullptr || (y_dtype == MTGR_I8 && d_y_scale == nullptr)))))
    return MTGR_ERR_INVALID_ARG;
  if (!aligned16(d_o) || !aligned16(d_u) || !aligned16(d_x) || !aligned16(d_h) || !aligned16(d_y))
    return MTGR_ERR_INVALID_ARG;
  BoundaryFwdArgs a{T, p->d, p->G, p->gate, p->eps, d_group_id, d_o, d_u, d_x, ld_o, ld_u,
                    p->post_gamma, p->post_beta, p->scale, p->pre_gamma, p->pre_beta, d_h, d_y, y_dtype,
                    d_y_scale};
  TimedScope tsc(MTGR_TIMER_GLN, as_stream(stream), T > 0 ? 1 : 0);
  return launch_boundary_fwd(a, o_dtype, x_dtype, as_stream(stream));
}

MTGR_API size_t mtgr_boundary_bwd_workspace_bytes(int32_t T, const mtgr_boundary_params* p) {
  if (boundary_check(p, T, MTGR_F32, MTGR_F32) != MTGR_OK) return 0;
  return boundary_bwd_ws_bytes(T, p->d, p->G);
}

MTGR_API int mtgr_boundary_bwd(const mtgr_boundary_params* p, int32_t T, const int8_t* d_group_id,
                               int32_t o_dtype, const void* d_o, int64_t ld_o, const void* d_u, int64_t ld_u,
                               int32_t x_dtype, const void* d_x, const void* d_dh, int32_t dy_dtype,
                               const void* d_dy, void* d_do, int64_t ld_do, void* d_du, int64_t ld_du,
                               void* d_dx, const mtgr_boundary_grads* grads, void* d_ws, size_t ws_bytes,
                               int32_t* d_status, mtgr_stream_t stream) {
  const int rc = boundary_check(p, T, o_dtype, x_dtype);
  if (rc != MTGR_OK) return rc;
  const bool gate = p->gate != MTGR_GATE_NONE, pre = p->pre_gamma != nullptr, post = p->post_gamma != nullptr;
  if (pre && dy_dtype != MTGR_F32 && dy_dtype != MTGR_BF16) return MTGR_ERR_UNSUPPORTED;
  if (!ld_ok(ld_o, p->d) || !ld_ok(ld_do, p->d) || (gate && (!ld_ok(ld_u, p->d) || !ld_ok(ld_du, p->d))))
    return MTGR_ERR_INVALID_ARG;
  if (grads == nullptr || (pre && (grads->pre_gamma == nullptr || grads->pre_beta == nullptr)) ||
      (post && (grads->post_gamma == nullptr || grads->post_beta == nullptr)) ||
      (p->scale != nullptr && grads->scale == nullptr))
    return MTGR_ERR_INVALID_ARG;
  if (T > 0 && (d_group_id == nullptr || d_o == nullptr || d_do == nullptr || d_dx == nullptr ||
                (gate && (d_u == nullptr || d_du == nullptr)) || (pre && (d_x == nullptr || d_dy == nullptr)) ||
                (!pre && d_dh == nullptr)))
    return MTGR_ERR_INVALID_ARG;
  if (!aligned16(d_o) || !aligned16(d_u) || !aligned16(d_x) || !aligned16(d_dh) || !aligned16(d_dy) ||
      !aligned16(d_do) || !aligned16(d_du) || !aligned16(d_dx) || !aligned16(grads->pre_gamma) ||
      !aligned16(grads->pre_beta) || !aligned16(grads->post_gamma) || !aligned16(grads->post_beta) ||
      !aligned16(grads->scale) || !aligned16(d_ws))
    return MTGR_ERR_INVALID_ARG;
  const size_t need = boundary_bwd_ws_bytes(T, p->d, p->G);
  if (ws_bytes < need) return MTGR_ERR_CAPACITY;
  if (need > 0 && d_ws == nullptr) return MTGR_ERR_INVALID_ARG;
  BoundaryBwdArgs a{T, p->d, p->G, p->gate, o_dtype, dy_dtype, p->eps, d_group_id, d_o, d_u, d_x, d_dh, d_dy,
                    ld_o, ld_u, ld_do, ld_du, p->post_gamma, p->post_beta, p->scale, p->pre_gamma, p->pre_beta,
                    d_do, d_du, d_dx, post ? grads->post_gamma : nullptr, post ? grads->post_beta : nullptr,
                    p->scale != nullptr ? grads->scale : nullptr, pre ? grads->pre_gamma : nullptr,
                    pre ? grads->pre_beta : nullptr, d_status, 0, 0, nullptr, nullptr};
  TimedScope tsc(MTGR_TIMER_BWD_GLN, as_stream(stream), T > 0 ? 2 : 1);
  return launch_boundary_bwd(a, x_dtype, d_ws, as_stream(stream));
}

MTGR_API int mtgr_quantize_rows(int32_t M, int32_t K, int32_t x_dtype, const void* d_x, int64_t ld_x,
                                int8_t* d_q, float* d_scale, mtgr_stream_t stream) {
  const int rc = quant_check(M, K, x_dtype, d_x, ld_x);
  if (rc != MTGR_OK) return rc;
  if (M > 0 && (d_q == nullptr || d_scale == nullptr)) return MTGR_ERR_INVALID_ARG;
  if (!aligned16(d_q) || is_operand(d_q, d_x, nullptr)) return MTGR_ERR_INVALID_ARG;
  TimedScope tsc(MTGR_TIMER_ROWS, as_stream(stream), M > 0 ? 1 : 0);
  return launch_quantize_rows(M, K, x_dtype, d_x, ld_x, d_q, d_scale, as_stream(stream));
}

MTGR_API int mtgr_gemm_i8(int32_t M, int32_t N, int32_t K, const int8_t* d_a, const float* d_a_scale,
                          const int8_t* d_b, const float* d_b_scale, const float* d_bias, int32_t epi,
                          const float* d_resid, int32_t q_cols, int32_t out_dtype, void* d_out,
                          int32_t* d_status, mtgr_stream_t stream) {
  const int rc = gemm_i8_check(M, N, K, d_b, d_b_scale, d_bias, epi, d_resid, q_cols, out_dtype, d_out);
  if (rc != MTGR_OK) return rc;
  if ((M > 0 && N > 0 && (d_a == nullptr || d_a_scale == nullptr)) || !aligned16(d_a)) return MTGR_ERR_INVALID_ARG;
  if (is_operand(d_out, d_a, d_b)) return MTGR_ERR_INVALID_ARG;
  if (!device_is_sm100()) return MTGR_ERR_UNSUPPORTED;
  TimedScope tsc(MTGR_TIMER_GEMM_QKVU, as_stream(stream), M > 0 && N > 0 ? 1 : 0);
  if (gemm_i8_is_few(M, N, K))
    return launch_gemm_i8_few(M, N, K, MTGR_I8, d_a, K, d_a_scale, d_b, d_b_scale, d_bias, epi, d_resid, q_cols,
                              out_dtype, d_out, d_status, as_stream(stream));
  return launch_gemm_i8(M, N, K, d_a, d_a_scale, d_b, d_b_scale, d_bias, epi, d_resid, q_cols, out_dtype, d_out,
                        d_status, as_stream(stream));
}

MTGR_API size_t mtgr_linear_i8_workspace_bytes(int32_t M, int32_t N, int32_t K) {
  if (M < 0 || N < 0 || K <= 0 || gemm_i8_is_few(M, N, K)) return 0;
  return align_up((size_t)M * (size_t)K, 256) + align_up((size_t)M * 4, 256);
}

MTGR_API int mtgr_linear_i8(int32_t M, int32_t N, int32_t K, int32_t x_dtype, const void* d_x, int64_t ld_x,
                            const int8_t* d_w, const float* d_w_scale, const float* d_bias, int32_t epi,
                            const float* d_resid, int32_t q_cols, int32_t out_dtype, void* d_out, void* d_ws,
                            size_t ws_bytes, int32_t* d_status, mtgr_stream_t stream) {
  int rc = gemm_i8_check(M, N, K, d_w, d_w_scale, d_bias, epi, d_resid, q_cols, out_dtype, d_out);
  if (rc != MTGR_OK) return rc;
  rc = quant_check(M, K, x_dtype, d_x, ld_x);
  if (rc != MTGR_OK) return rc;
  const size_t need = mtgr_linear_i8_workspace_bytes(M, N, K);
  if (ws_bytes < need) return MTGR_ERR_CAPACITY;
  if ((need > 0 && d_ws == nullptr) || !aligned16(d_ws)) return MTGR_ERR_INVALID_ARG;
  if (is_operand(d_out, d_x, d_w)) return MTGR_ERR_INVALID_ARG;
  if (!device_is_sm100()) return MTGR_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return MTGR_OK;
  if (need == 0) {
    TimedScope tsc(MTGR_TIMER_GEMM_QKVU, as_stream(stream), 1);
    return launch_gemm_i8_few(M, N, K, x_dtype, d_x, ld_x, nullptr, d_w, d_w_scale, d_bias, epi, d_resid, q_cols,
                              out_dtype, d_out, d_status, as_stream(stream));
  }
  int8_t* q = static_cast<int8_t*>(d_ws);
  float* sa = reinterpret_cast<float*>(static_cast<uint8_t*>(d_ws) + align_up((size_t)M * (size_t)K, 256));
  {
    TimedScope tsc(MTGR_TIMER_ROWS, as_stream(stream), 1);
    rc = launch_quantize_rows(M, K, x_dtype, d_x, ld_x, q, sa, as_stream(stream));
    if (rc != MTGR_OK) return rc;
  }
  TimedScope tsc(MTGR_TIMER_GEMM_QKVU, as_stream(stream), 1);
  return launch_gemm_i8(M, N, K, q, sa, d_w, d_w_scale, d_bias, epi, d_resid, q_cols, out_dtype, d_out, d_status,
                        as_stream(stream), true);
}

MTGR_API size_t mtgr_grad_clip_workspace_bytes(const mtgr_grad_tensor* h_grads, int32_t n) {
  if (grads_check(h_grads, n) != MTGR_OK) return 0;
  const size_t b = grad_clip_ws_bytes(h_grads, n);
  return b < 256 ? 256 : b;
}

MTGR_API int mtgr_grad_clip(const mtgr_grad_tensor* h_grads, int32_t n, float max_norm, float inv_scale,
                            float* d_norm, void* d_ws, size_t ws_bytes, int32_t* d_status,
                            mtgr_stream_t stream) {
  const int rc = grads_check(h_grads, n);
  if (rc != MTGR_OK) return rc;
  if (!(max_norm >= 0.0f) || !(inv_scale > 0.0f) || isinf(inv_scale) || d_norm == nullptr || d_status == nullptr)
    return MTGR_ERR_INVALID_ARG;
  if (ws_bytes < grad_clip_ws_bytes(h_grads, n)) return MTGR_ERR_CAPACITY;
  if (n > 0 && (d_ws == nullptr || !aligned16(d_ws))) return MTGR_ERR_INVALID_ARG;
  TimedScope tsc(MTGR_TIMER_BWD_ROWS, as_stream(stream), grad_clip_launches(h_grads, n));
  return launch_grad_clip(h_grads, n, max_norm, inv_scale, d_norm, d_ws, d_status, as_stream(stream));
}

}  // extern "C"
