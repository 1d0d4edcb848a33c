// The boundary between two blocks in one pass over the rows: the branch output o
// is normalised by group, gated by u, scaled and added to the residual stream x,
// and the next block's GroupLN reads the sum (GroupLN: fun-rec 7.3.3, the GLN
// formula, per token over d with the token's group's gamma and beta; the gate
// and the residual: summary page, Method, the block update equations):
//   n = GLN(o; post);  h = x + scale_g (.) n (.) f(u);  y = GLN(h; pre)
// with f none, u or silu(u), each norm and the scale optional, and y in fp32,
// bf16 or signed bytes with a scale per row.
//
// Backward, given dh (from the stream) and dy, with a = dy (.) gamma_pre and
// ohat, hhat the normalised rows, 1/sigma their rstd:
//   H = dh + (a - mean a - hhat mean(a hhat)) / sigma_h        (dx = H)
//   dscale += H n f;  dn = H scale f;  df = H scale n;  du = df f'(u)
//   b = dn gamma_post;  do = (b - mean b - ohat mean(b ohat)) / sigma_o
//   dgamma_pre += dy hhat, dbeta_pre += dy, dgamma_post += dn ohat, dbeta_post += dn
//
// Both are bound by HBM: at bf16 branch, fp32 stream and bf16 y the forward moves
// 14 bytes an element and the backward 22. Statistics, sums and gradients are
// held in fp32 (the sums over rows in fp32 per run of rows, then in fp64); the
// backward forms h again from x, o and u instead of reading a rounded one.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "ops.h"
#include "rowvec.cuh"

namespace mtgr {

namespace {

__device__ __forceinline__ float sigmoid_f32(float u) { return __fdividef(1.0f, 1.0f + __expf(-u)); }

// f(u); silu as u / (1 + e^-u): e^-u = inf gives -0, as the limit does
__device__ __forceinline__ void gate8(int gate, const float (&u)[8], float (&f)[8]) {
  if (gate == MTGR_GATE_SILU) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = __fdividef(u[e], 1.0f + __expf(-u[e]));
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = u[e];
  }
}

__device__ __forceinline__ int clamp_group(const int8_t* gid, int64_t t, int G) {
  const int g = gid[t];
  return g < 0 ? 0 : (g >= G ? G - 1 : g);
}

// ---------------------------------------------------------------- forward --
// One row per warp (d <= 1024) or per block of 256 (d <= 8192), VPL vectors of
// eight per thread; a row is read once and stays in registers through both norms.
template <typename TO, typename TX, bool BLOCK, int VPL>
__global__ void __launch_bounds__(256) boundary_fwd_kernel(BoundaryFwdArgs a) {
  __shared__ float part[BLOCK ? 2 : 1][1][32];
  Team<1, BLOCK> team(part);
  constexpr int TS = BLOCK ? 256 : 32;
  const int tl = threadIdx.x % TS;
  const int64_t t = BLOCK ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (t >= a.T) return;
  const int d = a.d, nv = d >> 3;
  const TO* o = static_cast<const TO*>(a.o) + t * a.ld_o;
  const TO* u = static_cast<const TO*>(a.u) + t * a.ld_u;
  const TX* x = static_cast<const TX*>(a.x) + t * d;
  Vec8<TO> ro[VPL], ru[VPL];
  Vec8<TX> rx[VPL];
#pragma unroll
  for (int k = 0; k < VPL; ++k) {
    const int vi = tl + TS * k;
    if (vi < nv) {
      ro[k].load(o + 8 * vi);
      rx[k].load(x + 8 * vi);
      if (a.gate != MTGR_GATE_NONE) ru[k].load(u + 8 * vi);
    }
  }
  const int g = clamp_group(a.gid, t, a.G);
  const float inv_d = 1.0f / (float)d;
  float mean = 0.f, rstd = 1.f;
  if (a.post_gamma != nullptr) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < VPL; ++k)
      if (tl + TS * k < nv) {
        float v[8];
        ro[k].unpack(v);
#pragma unroll
        for (int e = 0; e < 8; ++e) s += v[e];
      }
    mean = team.sum1(s) * inv_d;
    float q = 0.f;
#pragma unroll
    for (int k = 0; k < VPL; ++k)
      if (tl + TS * k < nv) {
        float v[8];
        ro[k].unpack(v);
#pragma unroll
        for (int e = 0; e < 8; ++e) q = fmaf(v[e] - mean, v[e] - mean, q);
      }
    rstd = 1.0f / sqrtf(team.sum1(q) * inv_d + a.eps);
  }
  float h[VPL][8];
  float s = 0.f;
#pragma unroll
  for (int k = 0; k < VPL; ++k) {
    const int vi = tl + TS * k;
    if (vi >= nv) continue;
    const int64_t pc = (int64_t)g * d + 8 * vi;
    float n[8];
    ro[k].unpack(n);
    if (a.post_gamma != nullptr) {
      float gm[8], bt[8];
      load8(a.post_gamma + pc, gm);
      load8(a.post_beta + pc, bt);
#pragma unroll
      for (int e = 0; e < 8; ++e) n[e] = fmaf((n[e] - mean) * rstd, gm[e], bt[e]);
    }
    if (a.gate != MTGR_GATE_NONE) {
      float uv[8], f[8];
      ru[k].unpack(uv);
      gate8(a.gate, uv, f);
#pragma unroll
      for (int e = 0; e < 8; ++e) n[e] *= f[e];
    }
    float xv[8];
    rx[k].unpack(xv);
    if (a.scale != nullptr) {
      float sc[8];
      load8(a.scale + pc, sc);
#pragma unroll
      for (int e = 0; e < 8; ++e) h[k][e] = fmaf(n[e], sc[e], xv[e]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) h[k][e] = n[e] + xv[e];
    }
    store8(static_cast<TX*>(a.h) + t * d + 8 * vi, h[k]);
#pragma unroll
    for (int e = 0; e < 8; ++e) s += h[k][e];
  }
  if (a.pre_gamma == nullptr) return;
  mean = team.sum1(s) * inv_d;
  float q = 0.f;
#pragma unroll
  for (int k = 0; k < VPL; ++k)
    if (tl + TS * k < nv) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        h[k][e] -= mean;
        q = fmaf(h[k][e], h[k][e], q);
      }
    }
  rstd = 1.0f / sqrtf(team.sum1(q) * inv_d + a.eps);
  uint32_t m = 0u;
#pragma unroll
  for (int k = 0; k < VPL; ++k) {
    const int vi = tl + TS * k;
    if (vi >= nv) continue;
    const int64_t pc = (int64_t)g * d + 8 * vi;
    float gm[8], bt[8];
    load8(a.pre_gamma + pc, gm);
    load8(a.pre_beta + pc, bt);
#pragma unroll
    for (int e = 0; e < 8; ++e) h[k][e] = fmaf(h[k][e] * rstd, gm[e], bt[e]);
    if (a.y_dtype == MTGR_F32) {
      store8(static_cast<float*>(a.y) + t * d + 8 * vi, h[k]);
    } else if (a.y_dtype == MTGR_BF16) {
      store8(static_cast<__nv_bfloat16*>(a.y) + t * d + 8 * vi, h[k]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(fabsf(h[k][e])));
    }
  }
  if (a.y_dtype != MTGR_I8) return;
  const RowScale rs = row_scale(team.max_bits(m));
  if (tl == 0) a.y_scale[t] = rs.s;
#pragma unroll
  for (int k = 0; k < VPL; ++k) {
    const int vi = tl + TS * k;
    if (vi < nv) *reinterpret_cast<uint2*>(static_cast<int8_t*>(a.y) + t * d + 8 * vi) = quant8(h[k], rs);
  }
}

template <typename TO, typename TX>
int launch_fwd_t(const BoundaryFwdArgs& a, cudaStream_t s) {
  if (a.d <= 1024) {
    const unsigned grid = (unsigned)(((int64_t)a.T + 7) / 8);
    switch ((a.d + 255) / 256) {
      case 1: boundary_fwd_kernel<TO, TX, false, 1><<<grid, 256, 0, s>>>(a); break;
      case 2: boundary_fwd_kernel<TO, TX, false, 2><<<grid, 256, 0, s>>>(a); break;
      case 3: boundary_fwd_kernel<TO, TX, false, 3><<<grid, 256, 0, s>>>(a); break;
      default: boundary_fwd_kernel<TO, TX, false, 4><<<grid, 256, 0, s>>>(a); break;
    }
  } else {
    switch ((a.d + 2047) / 2048) {
      case 1: boundary_fwd_kernel<TO, TX, true, 1><<<a.T, 256, 0, s>>>(a); break;
      case 2: boundary_fwd_kernel<TO, TX, true, 2><<<a.T, 256, 0, s>>>(a); break;
      case 3: boundary_fwd_kernel<TO, TX, true, 3><<<a.T, 256, 0, s>>>(a); break;
      default: boundary_fwd_kernel<TO, TX, true, 4><<<a.T, 256, 0, s>>>(a); break;
    }
  }
  return launch_status();
}

// --------------------------------------------------------------- backward --
// Gradient slots of the workspace, per team and group.
constexpr int kSlots = 5;
enum { kPreGamma = 0, kPreBeta = 1, kScale = 2, kPostGamma = 3, kPostBeta = 4 };

// A row's inputs as loaded.
template <typename TO, typename TX>
struct BwdRow {
  Vec8<TO> o, u;
  Vec8<TX> x, dh;
  float4 dy[2];  // raw: two float4 of fp32, or the first one as eight bf16
  int g;
};

// A team takes a contiguous run of rows (a user's segments are runs of one
// group, so the group seldom changes), one vector of eight a thread: a warp for
// d <= 256, several warps per block; above, a block of 32 ceil(d / 256) threads.
// The next row's inputs are loaded before the current row is computed. The
// parameter gradients gather in registers while the group stays the same; then
// they go to the team's own slots of the workspace (each thread its own columns:
// no atomics, and the same order of sums in every run).
// MAXT: the largest block of the form (0: a warp per team, 4 warps a block).
template <typename TO, typename TX, int MAXT>
__global__ void __launch_bounds__(MAXT == 0 ? 128 : MAXT, 1) boundary_bwd_kernel(BoundaryBwdArgs a) {
  constexpr bool BLOCK = MAXT != 0;
  __shared__ float part[BLOCK ? 2 : 1][2][32];
  Team<2, BLOCK> team(part);
  const int tl = BLOCK ? threadIdx.x : threadIdx.x & 31;
  const int64_t ti = BLOCK ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (ti >= a.teams) return;
  const int d = a.d;
  const bool on = tl < (d >> 3);
  const int c0 = 8 * tl;
  const int64_t t0 = ti * a.rows_per_team;
  const int64_t t1 = min((int64_t)a.T, t0 + a.rows_per_team);
  const bool post = a.post_gamma != nullptr, pre = a.pre_gamma != nullptr;
  const float inv_d = 1.0f / (float)d;
  float* slots = a.part + ti * a.G * kSlots * d + c0;

  float acc[kSlots][8];
#pragma unroll
  for (int i = 0; i < kSlots; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[i][e] = 0.f;
  uint32_t seen = 0u;
  int g_run = -1;
  bool range_bad = false;

  auto flush = [&]() {
    if (g_run < 0) return;
    if (on) {
      float* p = slots + (int64_t)g_run * kSlots * d;
      const bool add = (seen >> g_run) & 1u;
#pragma unroll
      for (int i = 0; i < kSlots; ++i) {
        float v[8];
        if (add) {
          load8(p + (int64_t)i * d, v);
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[i][e] += v[e];
        }
        store8(p + (int64_t)i * d, acc[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[i][e] = 0.f;
      }
    }
    seen |= 1u << g_run;
  };
  auto load_row = [&](int64_t t, BwdRow<TO, TX>& r) {
    r.o.zero();
    r.u.zero();
    r.x.zero();
    r.dh.zero();
    r.dy[0] = r.dy[1] = make_float4(0.f, 0.f, 0.f, 0.f);
    r.g = 0;
    if (t >= t1) return;
    r.g = clamp_group(a.gid, t, a.G);
    if (!on) return;
    r.o.load(static_cast<const TO*>(a.o) + t * a.ld_o + c0);
    if (a.gate != MTGR_GATE_NONE) r.u.load(static_cast<const TO*>(a.u) + t * a.ld_u + c0);
    if (pre) {
      r.x.load(static_cast<const TX*>(a.x) + t * d + c0);
      if (a.dy_dtype == MTGR_F32) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a.dy) + t * d + c0);
        r.dy[0] = p[0];
        r.dy[1] = p[1];
      } else {
        r.dy[0] = *reinterpret_cast<const float4*>(static_cast<const __nv_bfloat16*>(a.dy) + t * d + c0);
      }
    }
    if (a.dh != nullptr) r.dh.load(static_cast<const TX*>(a.dh) + t * d + c0);
  };

  BwdRow<TO, TX> cur;
  load_row(t0, cur);
  for (int64_t t = t0; t < t1; ++t) {
    BwdRow<TO, TX> nxt;
    load_row(t + 1, nxt);
    if (cur.g != g_run) {
      flush();
      g_run = cur.g;
    }
    const int64_t pc = (int64_t)cur.g * d + c0;
    // n and f again
    float oh[8], n[8], f[8], uv[8], gp[8], sc[8];
    float rstd_o = 1.f;
    cur.o.unpack(oh);
    if (post) {
      float s = 0.f, q = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) s += oh[e];
      const float mean = team.sum1(s) * inv_d;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        oh[e] = on ? oh[e] - mean : 0.f;
        q = fmaf(oh[e], oh[e], q);
      }
      rstd_o = 1.0f / sqrtf(team.sum1(q) * inv_d + a.eps);
      float bt[8];
      if (on) {
        load8(a.post_gamma + pc, gp);
        load8(a.post_beta + pc, bt);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) gp[e] = bt[e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        oh[e] *= rstd_o;
        n[e] = fmaf(oh[e], gp[e], bt[e]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) n[e] = oh[e];
    }
    cur.u.unpack(uv);
    if (a.gate != MTGR_GATE_NONE) {
      gate8(a.gate, uv, f);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = 1.f;
    }
    if (a.scale != nullptr && on) {
      load8(a.scale + pc, sc);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) sc[e] = 1.f;
    }
    // H: the gradient at h
    float H[8];
    cur.dh.unpack(H);
    if (pre) {
      float hh[8], s = 0.f, q = 0.f;
      cur.x.unpack(hh);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        hh[e] = fmaf(n[e] * f[e], sc[e], hh[e]);
        s += hh[e];
      }
      const float mean = team.sum1(on ? s : 0.f) * inv_d;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        hh[e] = on ? hh[e] - mean : 0.f;
        q = fmaf(hh[e], hh[e], q);
      }
      const float rstd_h = 1.0f / sqrtf(team.sum1(q) * inv_d + a.eps);
      float dy[8], gm[8];
      if (a.dy_dtype == MTGR_F32) {
        const float4 p0 = cur.dy[0], p1 = cur.dy[1];
        dy[0] = p0.x; dy[1] = p0.y; dy[2] = p0.z; dy[3] = p0.w;
        dy[4] = p1.x; dy[5] = p1.y; dy[6] = p1.z; dy[7] = p1.w;
      } else {
        const float w[4] = {cur.dy[0].x, cur.dy[0].y, cur.dy[0].z, cur.dy[0].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          dy[2 * k] = __uint_as_float(__float_as_uint(w[k]) << 16);
          dy[2 * k + 1] = __uint_as_float(__float_as_uint(w[k]) & 0xffff0000u);
        }
      }
      if (on) {
        load8(a.pre_gamma + pc, gm);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) gm[e] = 0.f;
      }
      float m[2] = {0.f, 0.f};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        hh[e] *= rstd_h;
        acc[kPreGamma][e] = fmaf(dy[e], hh[e], acc[kPreGamma][e]);
        acc[kPreBeta][e] += dy[e];
        dy[e] *= gm[e];
        m[0] += dy[e];
        m[1] = fmaf(dy[e], hh[e], m[1]);
      }
      team.sum(m);
      const float m0 = m[0] * inv_d, m1 = m[1] * inv_d;
#pragma unroll
      for (int e = 0; e < 8; ++e) H[e] = fmaf(rstd_h, dy[e] - m0 - hh[e] * m1, H[e]);
    }
    if (on) store8(static_cast<TX*>(a.dx) + t * d + c0, H);
    float b[8], m[2] = {0.f, 0.f};
    {
      float du[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float p = H[e] * sc[e];
        acc[kScale][e] = fmaf(H[e], n[e] * f[e], acc[kScale][e]);
        b[e] = p * f[e];  // dn
        du[e] = p * n[e];
        acc[kPostGamma][e] = fmaf(b[e], oh[e], acc[kPostGamma][e]);
        acc[kPostBeta][e] += b[e];
      }
      if (a.gate == MTGR_GATE_SILU) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float sg = sigmoid_f32(uv[e]);
          du[e] *= fmaf(f[e], 1.0f - sg, sg);  // sigmoid(u) (1 + u (1 - sigmoid(u)))
        }
      }
      if (a.gate != MTGR_GATE_NONE && on) {
        store8(static_cast<TO*>(a.du) + t * a.ld_du + c0, du);
        if (sizeof(TO) == 2 && a.o_dtype == MTGR_F16)
#pragma unroll
          for (int e = 0; e < 8; ++e) range_bad |= fabsf(du[e]) > 65504.f;
      }
    }
    if (post) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        b[e] *= gp[e];
        m[0] += b[e];
        m[1] = fmaf(b[e], oh[e], m[1]);
      }
      team.sum(m);
      const float m0 = m[0] * inv_d, m1 = m[1] * inv_d;
#pragma unroll
      for (int e = 0; e < 8; ++e) b[e] = rstd_o * (b[e] - m0 - oh[e] * m1);
    }
    if (on) {
      store8(static_cast<TO*>(a.d_o) + t * a.ld_do + c0, b);
      if (sizeof(TO) == 2 && a.o_dtype == MTGR_F16)
#pragma unroll
        for (int e = 0; e < 8; ++e) range_bad |= fabsf(b[e]) > 65504.f;
    }
    cur = nxt;
  }
  flush();
  if (tl == 0) a.seen[ti] = seen;
  if (range_bad) set_status(a.status, MTGR_ERR_RANGE);
}

// The parameter gradients: each of the G * 5 * d columns summed over the teams
// that saw its group, a block per 128 columns, 16 warps over the teams in a
// fixed order, in fp64.
__global__ void __launch_bounds__(512) boundary_bwd_reduce_kernel(BoundaryBwdArgs a) {
  __shared__ double red[16][32][4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t n = (int64_t)a.G * kSlots * a.d;
  const int64_t c = ((int64_t)blockIdx.x * 32 + lane) * 4;  // d % 8 == 0: one slot and group per 4 columns
  const int gs = c < n ? (int)(c / a.d) : 0;
  const int g = gs / kSlots, slot = gs % kSlots;
  double s[4] = {0.0, 0.0, 0.0, 0.0};
  if (c < n) {
#pragma unroll 4
    for (int i = warp; i < a.teams; i += 16) {
      if ((a.seen[i] >> g) & 1u) {
        const float4 v = *reinterpret_cast<const float4*>(a.part + i * n + c);
        s[0] += v.x; s[1] += v.y; s[2] += v.z; s[3] += v.w;
      }
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) red[warp][lane][k] = s[k];
  __syncthreads();
  if (warp != 0 || c >= n) return;
#pragma unroll
  for (int w = 1; w < 16; ++w)
#pragma unroll
    for (int k = 0; k < 4; ++k) s[k] += red[w][lane][k];
  float* out = slot == kPreGamma    ? a.g_pre_gamma
               : slot == kPreBeta   ? a.g_pre_beta
               : slot == kScale     ? a.g_scale
               : slot == kPostGamma ? a.g_post_gamma
                                    : a.g_post_beta;
  if (out == nullptr) return;
  *reinterpret_cast<float4*>(out + (int64_t)g * a.d + (c - (int64_t)gs * a.d)) =
      make_float4((float)s[0], (float)s[1], (float)s[2], (float)s[3]);
}

template <typename TO, typename TX>
int launch_bwd_t(const BoundaryBwdArgs& a, cudaStream_t s) {
  if (a.teams > 0) {
    const int threads = 32 * ((a.d + 255) / 256);
    if (a.d <= 256) {
      boundary_bwd_kernel<TO, TX, 0><<<(a.teams + 3) / 4, 128, 0, s>>>(a);
    } else if (a.d <= 2048) {
      boundary_bwd_kernel<TO, TX, 256><<<a.teams, threads, 0, s>>>(a);
    } else {
      boundary_bwd_kernel<TO, TX, 1024><<<a.teams, threads, 0, s>>>(a);
    }
    const int rc = launch_status();
    if (rc != MTGR_OK) return rc;
  }
  const int64_t n = (int64_t)a.G * kSlots * a.d;
  boundary_bwd_reduce_kernel<<<(unsigned)((n + 127) / 128), 512, 0, s>>>(a);
  return launch_status();
}

}  // namespace

// Teams of the backward: as many as are resident at once (register-bound: 16
// warps an SM), at least 4 rows each, and at most 256 MB of gradient slots.
int32_t boundary_bwd_teams(int32_t T, int32_t d, int32_t G) {
  if (T <= 0) return 0;
  const int warps = (d + 255) / 256;
  int64_t teams = (int64_t)device_sm_count() * (16 / warps > 0 ? 16 / warps : 1);
  const int64_t slot_bytes = (int64_t)G * kSlots * d * 4;
  const int64_t most = (256ll << 20) / slot_bytes;
  if (teams > most) teams = most > 0 ? most : 1;
  const int64_t by_rows = ((int64_t)T + 3) / 4;
  if (teams > by_rows) teams = by_rows;
  const int64_t rows = ((int64_t)T + teams - 1) / teams;
  return (int32_t)(((int64_t)T + rows - 1) / rows);
}

size_t boundary_bwd_ws_bytes(int32_t T, int32_t d, int32_t G) {
  const size_t teams = (size_t)boundary_bwd_teams(T, d, G);
  return align_up(teams * 4, 256) + teams * G * kSlots * d * 4;
}

int launch_boundary_fwd(const BoundaryFwdArgs& a, int32_t o_dtype, int32_t x_dtype, cudaStream_t s) {
  if (a.T == 0) return MTGR_OK;
  if (x_dtype == MTGR_F32) {
    if (o_dtype == MTGR_F32) return launch_fwd_t<float, float>(a, s);
    if (o_dtype == MTGR_BF16) return launch_fwd_t<__nv_bfloat16, float>(a, s);
    if (o_dtype == MTGR_F16) return launch_fwd_t<__half, float>(a, s);
  } else if (x_dtype == MTGR_BF16) {
    if (o_dtype == MTGR_F32) return launch_fwd_t<float, __nv_bfloat16>(a, s);
    if (o_dtype == MTGR_BF16) return launch_fwd_t<__nv_bfloat16, __nv_bfloat16>(a, s);
    if (o_dtype == MTGR_F16) return launch_fwd_t<__half, __nv_bfloat16>(a, s);
  }
  return MTGR_ERR_UNSUPPORTED;
}

int launch_boundary_bwd(BoundaryBwdArgs a, int32_t x_dtype, void* ws, cudaStream_t s) {
  a.teams = boundary_bwd_teams(a.T, a.d, a.G);
  a.rows_per_team = a.teams > 0 ? (a.T + a.teams - 1) / a.teams : 0;
  a.seen = static_cast<uint32_t*>(ws);
  a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + align_up((size_t)a.teams * 4, 256));
  if (x_dtype == MTGR_F32) {
    if (a.o_dtype == MTGR_F32) return launch_bwd_t<float, float>(a, s);
    if (a.o_dtype == MTGR_BF16) return launch_bwd_t<__nv_bfloat16, float>(a, s);
    if (a.o_dtype == MTGR_F16) return launch_bwd_t<__half, float>(a, s);
  } else if (x_dtype == MTGR_BF16) {
    if (a.o_dtype == MTGR_F32) return launch_bwd_t<float, __nv_bfloat16>(a, s);
    if (a.o_dtype == MTGR_BF16) return launch_bwd_t<__nv_bfloat16, __nv_bfloat16>(a, s);
    if (a.o_dtype == MTGR_F16) return launch_bwd_t<__half, __nv_bfloat16>(a, s);
  }
  return MTGR_ERR_UNSUPPORTED;
}

}  // namespace mtgr
