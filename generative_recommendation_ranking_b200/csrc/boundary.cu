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

// A row's inputs wait in shared memory: each thread copies its own eight values of
// every input up to two rows ahead (cp.async) and reads back only those, so no barrier
// is needed, and the registers hold the sums instead. Stage layout: per thread
// o, u (16 or 32 bytes), x, dh, dy; a thread's 16-byte pieces lie THREADS * 16
// bytes apart, so that a warp's accesses fall in different banks.
template <typename T>
constexpr int kPieces = sizeof(T) / 2;  // 16-byte pieces of eight values: 1 or 2

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 shared16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}

template <typename T>
__device__ __forceinline__ void copy8(uint32_t dst, uint32_t step, const T* src) {
#pragma unroll
  for (int i = 0; i < kPieces<T>; ++i) copy16(dst + i * step, reinterpret_cast<const char*>(src) + 16 * i);
}
__device__ __forceinline__ void unpack16(const uint4& a, float (&v)[8], __nv_bfloat16) {
  Vec8<__nv_bfloat16> r;
  r.a = a;
  r.unpack(v);
}
__device__ __forceinline__ void unpack16(const uint4& a, float (&v)[8], __half) {
  Vec8<__half> r;
  r.a = a;
  r.unpack(v);
}
template <typename T>
__device__ __forceinline__ void read8(uint32_t src, uint32_t step, float (&v)[8]) {
  if constexpr (sizeof(T) == 4) {
    const uint4 a = shared16(src), b = shared16(src + step);
    v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y); v[2] = __uint_as_float(a.z); v[3] = __uint_as_float(a.w);
    v[4] = __uint_as_float(b.x); v[5] = __uint_as_float(b.y); v[6] = __uint_as_float(b.z); v[7] = __uint_as_float(b.w);
  } else {
    unpack16(shared16(src), v, T());
  }
}

// Warps of a row's team.
inline int bwd_warps(int d) {
  const int w = (d + 255) / 256;
  return w <= 4 ? w : (w <= 8 ? 8 : (w <= 16 ? 16 : 32));
}

// Rows in flight beside the one computed: two where 16 warps' stages fit in an SM.
template <typename TO, int WARPS>
constexpr int kAhead = WARPS == 32 ? 0 : (WARPS == 16 || sizeof(TO) == 4 ? 1 : 2);

template <typename TO, typename TX>
constexpr int kRowBytes = 16 * (2 * kPieces<TO> + 2 * kPieces<TX> + 2);

// Sums over a team: a warp, or a block of WARPS warps that meet in shared memory
// (partials in two slots used in turn, so that one barrier a sum is enough).
template <int WARPS>
struct Sums {
  float2* part;  // [2][WARPS]
  int turn = 0;
  __device__ __forceinline__ float2 operator()(float a, float b) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    return meet(make_float2(a, b));
  }
  __device__ __forceinline__ float operator()(float a) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    return meet(make_float2(a, 0.f)).x;
  }
  __device__ __forceinline__ float2 meet(float2 v) {
    if constexpr (WARPS > 1) {
      float2* p = part + turn * WARPS;
      if ((threadIdx.x & 31) == 0) p[threadIdx.x >> 5] = v;
      __syncthreads();
      v = p[0];
#pragma unroll
      for (int w = 1; w < WARPS; ++w) {
        v.x += p[w].x;
        v.y += p[w].y;
      }
      turn ^= 1;
    }
    return v;
  }
};

// A team takes a contiguous run of rows (a user's segments are runs of one
// group, so the group seldom changes), one vector of eight a thread: a warp for
// d <= 256, four to a block; above, a block of WARPS = ceil(d / 256) warps (rounded
// up to a power of two past four). The parameter gradients gather in registers
// while the group stays the same; then they go to the team's own slots of the
// workspace (each thread its own columns: no atomics, and the same order of sums
// in every run).
template <typename TO, typename TX, int WARPS>
__global__ void __launch_bounds__(WARPS == 1 ? 128 : 32 * WARPS, WARPS <= 2 ? 8 / (WARPS == 1 ? 2 : 1) : (WARPS <= 16 ? 16 / WARPS : 1))
    boundary_bwd_kernel(BoundaryBwdArgs a) {
  constexpr int AHEAD = kAhead<TO, WARPS>;
  extern __shared__ uint4 smem[];
  __shared__ float2 part[2 * WARPS];
  Sums<WARPS> sums{part};
  constexpr bool BLOCK = WARPS > 1;
  const int tl = BLOCK ? threadIdx.x : threadIdx.x & 31;
  const int64_t ti = BLOCK ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (ti >= a.teams) return;
  const int d = a.d;
  const bool on = tl < (d >> 3);
  const int c0 = 8 * tl;
  const int64_t t0 = ti * a.rows_per_team;
  const int rows = (int)min((int64_t)a.rows_per_team, (int64_t)a.T - t0);
  const bool post = a.post_gamma != nullptr, pre = a.pre_gamma != nullptr, gate = a.gate != MTGR_GATE_NONE;
  const float inv_d = 1.0f / (float)d;
  float* slots = a.part + ti * a.G * kSlots * d + c0;
  // this thread's pieces: stage s at base + s * stage, input pieces `step` apart
  const uint32_t step = blockDim.x * 16, stage = kRowBytes<TO, TX> / 16 * step;
  const uint32_t base = (uint32_t)__cvta_generic_to_shared(smem) + threadIdx.x * 16;
  constexpr int PO = kPieces<TO>, PX = kPieces<TX>;

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
  auto copy_row = [&](int r, int s) {
    if (on && r < rows) {
      const int64_t t = t0 + r;
      const uint32_t at = base + s * stage;
      copy8(at, step, static_cast<const TO*>(a.o) + t * a.ld_o + c0);
      if (gate) copy8(at + PO * step, step, static_cast<const TO*>(a.u) + t * a.ld_u + c0);
      if (a.dh != nullptr) copy8(at + (2 * PO + PX) * step, step, static_cast<const TX*>(a.dh) + t * d + c0);
      if (pre) {
        copy8(at + 2 * PO * step, step, static_cast<const TX*>(a.x) + t * d + c0);
        if (a.dy_dtype == MTGR_F32)
          copy8(at + (2 * PO + 2 * PX) * step, step, static_cast<const float*>(a.dy) + t * d + c0);
        else
          copy8(at + (2 * PO + 2 * PX) * step, step, static_cast<const __nv_bfloat16*>(a.dy) + t * d + c0);
      }
    }
    copy_commit();
  };

#pragma unroll
  for (int r = 0; r < AHEAD; ++r) copy_row(r, r);
  int g = rows > 0 ? clamp_group(a.gid, t0, a.G) : 0, s = 0;
  for (int r = 0; r < rows; ++r) {
    copy_row(r + AHEAD, s == 0 ? AHEAD : s - 1);  // stage (s + AHEAD) mod (AHEAD + 1)
    const int g_next = r + 1 < rows ? clamp_group(a.gid, t0 + r + 1, a.G) : 0;
    copy_wait<AHEAD>();
    const uint32_t at = base + s * stage;
    if (g != g_run) {
      flush();
      g_run = g;
    }
    const int64_t t = t0 + r, pc = (int64_t)g * d + c0;
    // n and f again (what is past d is 0, so that it adds nothing to a sum)
    float oh[8] = {}, n[8], f[8], gp[8] = {}, sc[8];
    float rstd_o = 1.f;
    if (on) read8<TO>(at, step, oh);
    if (post) {
      float q = 0.f, m = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) m += oh[e];
      m = sums(m) * inv_d;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        oh[e] = on ? oh[e] - m : 0.f;
        q = fmaf(oh[e], oh[e], q);
      }
      rstd_o = 1.0f / sqrtf(sums(q) * inv_d + a.eps);
      float bt[8] = {};
      if (on) {
        load8(a.post_gamma + pc, gp);
        load8(a.post_beta + pc, bt);
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
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = 1.f;
    if (gate) {
      float uv[8] = {};
      if (on) read8<TO>(at + PO * step, step, uv);
      gate8(a.gate, uv, f);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) sc[e] = 1.f;
    if (a.scale != nullptr && on) load8(a.scale + pc, sc);
    // H: the gradient at h
    float H[8] = {};
    if (pre) {
      float hh[8] = {}, m = 0.f, q = 0.f;
      if (on) read8<TX>(at + 2 * PO * step, step, hh);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        hh[e] = fmaf(n[e] * f[e], sc[e], hh[e]);
        m += hh[e];
      }
      m = sums(on ? m : 0.f) * inv_d;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        hh[e] = on ? hh[e] - m : 0.f;
        q = fmaf(hh[e], hh[e], q);
      }
      const float rstd_h = 1.0f / sqrtf(sums(q) * inv_d + a.eps);
      float dy[8] = {}, gm[8] = {};
      if (on) {
        if (a.dy_dtype == MTGR_F32) read8<float>(at + (2 * PO + 2 * PX) * step, step, dy);
        else read8<__nv_bfloat16>(at + (2 * PO + 2 * PX) * step, step, dy);
        load8(a.pre_gamma + pc, gm);
      }
      float m0 = 0.f, m1 = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        hh[e] *= rstd_h;
        acc[kPreGamma][e] = fmaf(dy[e], hh[e], acc[kPreGamma][e]);
        acc[kPreBeta][e] += dy[e];
        dy[e] *= gm[e];
        m0 += dy[e];
        m1 = fmaf(dy[e], hh[e], m1);
      }
      const float2 ms = sums(m0, m1);
      m0 = ms.x * inv_d;
      m1 = ms.y * inv_d;
#pragma unroll
      for (int e = 0; e < 8; ++e) H[e] = rstd_h * (dy[e] - m0 - hh[e] * m1);
    }
    if (a.dh != nullptr && on) {
      float dh[8];
      read8<TX>(at + (2 * PO + PX) * step, step, dh);
#pragma unroll
      for (int e = 0; e < 8; ++e) H[e] += dh[e];
    }
    if (on) store8(static_cast<TX*>(a.dx) + t * d + c0, H);
    float b[8], m0 = 0.f, m1 = 0.f;
    if (gate) {
      float du[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) du[e] = H[e] * sc[e] * n[e];
      if (a.gate == MTGR_GATE_SILU && on) {
        float uv[8];
        read8<TO>(at + PO * step, step, uv);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float sg = sigmoid_f32(uv[e]);
          du[e] *= fmaf(f[e], 1.0f - sg, sg);  // sigmoid(u) (1 + u (1 - sigmoid(u)))
        }
      }
      if (on) {
        store8(static_cast<TO*>(a.du) + t * a.ld_du + c0, du);
        if (sizeof(TO) == 2 && a.o_dtype == MTGR_F16)
#pragma unroll
          for (int e = 0; e < 8; ++e) range_bad |= fabsf(du[e]) > 65504.f;
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float hf = H[e] * f[e];
      acc[kScale][e] = fmaf(hf, n[e], acc[kScale][e]);
      b[e] = hf * sc[e];  // dn
      acc[kPostGamma][e] = fmaf(b[e], oh[e], acc[kPostGamma][e]);
      acc[kPostBeta][e] += b[e];
      b[e] = post ? b[e] * gp[e] : b[e];
      m0 += b[e];
      m1 = fmaf(b[e], oh[e], m1);
    }
    if (post) {
      const float2 ms = sums(m0, m1);
      m0 = ms.x * inv_d;
      m1 = ms.y * inv_d;
#pragma unroll
      for (int e = 0; e < 8; ++e) b[e] = rstd_o * (b[e] - m0 - oh[e] * m1);
    }
    if (on) {
      store8(static_cast<TO*>(a.d_o) + t * a.ld_do + c0, b);
      if (sizeof(TO) == 2 && a.o_dtype == MTGR_F16)
#pragma unroll
        for (int e = 0; e < 8; ++e) range_bad |= fabsf(b[e]) > 65504.f;
    }
    g = g_next;
    s = s == AHEAD ? 0 : s + 1;
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

template <typename TO, typename TX, int WARPS>
int launch_bwd_w(const BoundaryBwdArgs& a, cudaStream_t s) {
  const int threads = WARPS == 1 ? 128 : 32 * WARPS;
  const int bytes = threads * (kAhead<TO, WARPS> + 1) * kRowBytes<TO, TX>;
  auto kern = boundary_bwd_kernel<TO, TX, WARPS>;
  if (bytes > 40 * 1024 &&  // 48 KB without asking, some of it static
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
    return MTGR_ERR_CUDA;
  kern<<<WARPS == 1 ? (a.teams + 3) / 4 : a.teams, threads, bytes, s>>>(a);
  return launch_status();
}

template <typename TO, typename TX>
int launch_bwd_t(const BoundaryBwdArgs& a, cudaStream_t s) {
  if (a.teams > 0) {
    int rc = MTGR_OK;
    switch (bwd_warps(a.d)) {
      case 1: rc = launch_bwd_w<TO, TX, 1>(a, s); break;
      case 2: rc = launch_bwd_w<TO, TX, 2>(a, s); break;
      case 3: rc = launch_bwd_w<TO, TX, 3>(a, s); break;
      case 4: rc = launch_bwd_w<TO, TX, 4>(a, s); break;
      case 8: rc = launch_bwd_w<TO, TX, 8>(a, s); break;
      case 16: rc = launch_bwd_w<TO, TX, 16>(a, s); break;
      default: rc = launch_bwd_w<TO, TX, 32>(a, s); break;
    }
    if (rc != MTGR_OK) return rc;
  }
  const int64_t n = (int64_t)a.G * kSlots * a.d;
  boundary_bwd_reduce_kernel<<<(unsigned)((n + 127) / 128), 512, 0, s>>>(a);
  return launch_status();
}

}  // namespace

// Teams of the backward: as many as are resident at once (16 warps an SM, by
// registers), at least 4 rows each, and at most 256 MB of gradient slots.
int32_t boundary_bwd_teams(int32_t T, int32_t d, int32_t G) {
  if (T <= 0) return 0;
  const int warps = bwd_warps(d);
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
