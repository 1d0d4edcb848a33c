// The boundary between two blocks in one pass over the rows: the branch output o
// is normalised by group, gated by u, scaled and added to the residual stream x,
// and the next block's GroupLN reads the sum (GroupLN: fun-rec 7.3.3, the GLN
// formula, per token over d with the token's group's gamma and beta):
//   n = GLN(o; post);  h = x + scale_g (.) n (.) f(u);  y = GLN(h; pre)
// with f none, u or silu(u), each norm and the scale optional, and y in fp32,
// bf16 or signed bytes with a scale per row. Between this library's blocks, which gate
// inside their second norm, f and the post norm are absent: h = x + o, y = GLN(h).
//
// Backward, given dh (from the stream) and dy, with a = dy (.) gamma_pre and
// ohat, hhat the normalised rows, 1/sigma their rstd:
//   H = dh + (a - mean a - hhat mean(a hhat)) / sigma_h        (dx = H)
//   dscale += H n f;  dn = H scale f;  df = H scale n;  du = df f'(u)
//   b = dn gamma_post;  do = (b - mean b - ohat mean(b ohat)) / sigma_o
//   dgamma_pre += dy hhat, dbeta_pre += dy, dgamma_post += dn ohat, dbeta_post += dn
//
// At bf16 branch, fp32 stream and bf16 y the forward moves 14 bytes an element, which
// bounds it, and the backward 22; that one is bound by its instructions' latency from
// d = 256 on, at two warps a scheduler (0.70 of the copy rate). Statistics, sums and gradients are
// held in fp32; the backward forms h again from x, o and u instead of reading a rounded
// one. A parameter's gradient adds up in fp32 over a team's run of rows (registers; 169
// rows at 200003 x 512, about T / 50 with 32 groups of 8192 columns, whose slots are limited),
// then in fp64 over the teams.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "ops.h"
#include "row_runs.h"
#include "rowvec.cuh"

namespace mtgr {

namespace {

// e^-u by __expf, within 2 + 1.2 |u| ulp: far below a rounding of a bf16 or f16 branch, a few
// ulp of an fp32 one. The quotient by __fdividef, within 2 ulp, and 0 where 1 + e^-u is
// beyond 2^126 (|silu| below 1e-36).
__device__ __forceinline__ float sigmoid_f32(float u) { return __fdividef(1.0f, 1.0f + __expf(-u)); }

// silu as u / (1 + e^-u): e^-u = inf gives -0, as the limit does
__device__ __forceinline__ float silu_f32(float u) { return __fdividef(u, 1.0f + __expf(-u)); }

__device__ __forceinline__ bool beyond_f16(const f2 (&v)[4]) {
  float m = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f = unpair2(v[k]);
    m = fmaxf(m, fmaxf(fabsf(f.x), fabsf(f.y)));
  }
  return m > 65504.f;
}

__device__ __forceinline__ int clamp_group(const int8_t* gid, int64_t t, int G) {
  const int g = gid[t];
  return g < 0 ? 0 : (g >= G ? G - 1 : g);
}

// 16-byte pieces of eight values: 1 or 2
template <typename T>
constexpr int kPieces = sizeof(T) / 2;

template <typename T>
__device__ __forceinline__ void fetch8(bool on, const T* p, uint4 (&r)[kPieces<T>]) {
#pragma unroll
  for (int i = 0; i < kPieces<T>; ++i)
    r[i] = on ? reinterpret_cast<const uint4*>(p)[i] : make_uint4(0u, 0u, 0u, 0u);
}
__device__ __forceinline__ void zero8(f2 (&v)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = 0ull;
}
__device__ __forceinline__ void load_param(bool on, const float* p, f2 (&v)[4]) {
  uint4 r[2];
  fetch8<float>(on, p, r);
  to_pairs(r[0], r[1], v, 0.f);
}

// Sums over a team: LANES lanes of a warp, or a block of WARPS warps that meet in
// shared memory (partials in two slots used in turn, so that one barrier a sum is
// enough).
template <int WARPS, int LANES>
struct Sums {
  static_assert(WARPS == 1 || LANES == 32, "a block's team is whole warps");
  float* part;  // [2][WARPS][2]
  int turn = 0;
  __device__ __forceinline__ float operator()(float a) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    if constexpr (WARPS > 1) {
      float* p = part + turn * 2 * WARPS;
      if ((threadIdx.x & 31) == 0) p[threadIdx.x >> 5] = a;
      __syncthreads();
      a = p[0];
#pragma unroll
      for (int w = 1; w < WARPS; ++w) a += p[w];
      turn ^= 1;
    }
    return a;
  }
  // two sums for half the exchanges: the lanes' halves swap one value each, and
  // each half adds up the other value
  __device__ __forceinline__ float2 operator()(float a, float b) {
    constexpr int HALF = LANES / 2;
    const bool low = (threadIdx.x & HALF) == 0;
    const float give = low ? b : a;
    float keep = low ? a : b;
    keep += __shfl_xor_sync(0xffffffffu, give, HALF);
#pragma unroll
    for (int o = HALF / 2; o > 0; o >>= 1) keep += __shfl_xor_sync(0xffffffffu, keep, o);
    float2 v;
    if constexpr (WARPS > 1) {
      float* p = part + turn * 2 * WARPS;
      if ((threadIdx.x & 15) == 0) p[2 * (threadIdx.x >> 5) + (low ? 0 : 1)] = keep;
      __syncthreads();
      v = make_float2(p[0], p[1]);
#pragma unroll
      for (int w = 1; w < WARPS; ++w) {
        v.x += p[2 * w];
        v.y += p[2 * w + 1];
      }
      turn ^= 1;
    } else {
      const float other = __shfl_xor_sync(0xffffffffu, keep, HALF);
      v = low ? make_float2(keep, other) : make_float2(other, keep);
    }
    return v;
  }
  // maximum of non-negative values by their bits: a NaN is above every number
  // and an infinity, so it is not lost
  __device__ __forceinline__ uint32_t max_bits(uint32_t a) {
    if constexpr (LANES < 32) {
#pragma unroll
      for (int o = LANES / 2; o > 0; o >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
    } else {
      a = __reduce_max_sync(0xffffffffu, a);
    }
    if constexpr (WARPS > 1) {
      float* p = part + turn * 2 * WARPS;
      if ((threadIdx.x & 31) == 0) p[threadIdx.x >> 5] = __uint_as_float(a);
      __syncthreads();
      a = __float_as_uint(p[0]);
#pragma unroll
      for (int w = 1; w < WARPS; ++w) a = max(a, __float_as_uint(p[w]));
      turn ^= 1;
    }
    return a;
  }
};

// ---------------------------------------------------------------- forward --
// A row per team: LANES lanes of a warp (8 for d <= 64, 16 for d <= 128, 32 up to 512),
// or a block of WARPS warps, VPL vectors of eight columns a thread; a row is read once
// and stays in registers through both norms. Two vectors a thread (at 65537 x 1024 with int8 y, one warp a
// row with four took 226 us, two warps with two 171), small blocks, so that rows of
// different blocks are in different steps (200003 x 512: 261 us in blocks of eight
// rows, 237 of two), and 28 warps an SM by registers.
template <typename TO, typename TX, int WARPS, int LANES, int VPL>
__global__ void __launch_bounds__(WARPS == 1 ? 64 : 32 * WARPS, VPL == 2 ? 28 / (WARPS < 2 ? 2 : WARPS) : 1)
    boundary_fwd_kernel(BoundaryFwdArgs a) {
  constexpr bool BLOCK = WARPS > 1;
  __shared__ float part[BLOCK ? 4 * WARPS : 1];
  Sums<WARPS, LANES> sums{part};
  const int tl = BLOCK ? threadIdx.x : threadIdx.x % LANES;
  const int64_t t = BLOCK ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * (64 / LANES) + threadIdx.x / LANES;
  if (LANES == 32 && t >= a.T) return;
  const int d = t < a.T ? a.d : 0;  // a team without a row has no columns, but goes along
  constexpr int VSTEP = 8 * LANES * WARPS;  // columns between a thread's vectors
  const int c0 = 8 * tl;
  const bool gate = a.gate != MTGR_GATE_NONE;
  uint4 ro[VPL][kPieces<TO>], ru[VPL][kPieces<TO>], rx[VPL][kPieces<TX>];
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const int c = c0 + j * VSTEP;
    const bool on = c < d;
    fetch8<TO>(on, static_cast<const TO*>(a.o) + t * a.ld_o + c, ro[j]);
    fetch8<TX>(on, static_cast<const TX*>(a.x) + t * d + c, rx[j]);
    fetch8<TO>(on && gate, static_cast<const TO*>(a.u) + t * a.ld_u + c, ru[j]);
  }
  const int g = d > 0 ? clamp_group(a.gid, t, a.G) : 0;
  const int64_t pc = (int64_t)g * d + c0;
  const float inv_d = 1.0f / (float)a.d;
  f2 h[VPL][4], v[4], w[4];
#pragma unroll
  for (int j = 0; j < VPL; ++j) to_pairs(ro[j][0], ro[j][kPieces<TO> - 1], h[j], TO());
  // the rows' mean and 1 / sigma; h becomes the centred row (0 past d)
  auto centre = [&]() {
    f2 q = 0ull;
#pragma unroll
    for (int j = 0; j < VPL; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) q = add2(q, h[j][k]);
    const f2 m = both(-sums(sum_of(q)) * inv_d);
    float sq = 0.f;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      q = 0ull;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        h[j][k] = add2(h[j][k], m);
        q = fma2(h[j][k], h[j][k], q);
      }
      sq += c0 + j * VSTEP < d ? sum_of(q) : 0.f;
    }
    return rsqrtf(sums(sq) * inv_d + a.eps);
  };
  const bool post = a.post_gamma != nullptr;
  const float rstd_o = post ? centre() : 1.f;
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const int c = c0 + j * VSTEP;
    const bool on = c < d;
    if (post) {
      load_param(on, a.post_gamma + pc + j * VSTEP, v);
      load_param(on, a.post_beta + pc + j * VSTEP, w);
#pragma unroll
      for (int k = 0; k < 4; ++k) h[j][k] = fma2(mul2(h[j][k], both(rstd_o)), v[k], w[k]);
    }
    if (gate) {
      to_pairs(ru[j][0], ru[j][kPieces<TO> - 1], v, TO());
      if (a.gate == MTGR_GATE_SILU) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 u = unpair2(v[k]);
          v[k] = pair2(silu_f32(u.x), silu_f32(u.y));
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) h[j][k] = mul2(h[j][k], v[k]);
    }
    to_pairs(rx[j][0], rx[j][kPieces<TX> - 1], v, TX());
    if (a.scale != nullptr) {
      load_param(on, a.scale + pc + j * VSTEP, w);
#pragma unroll
      for (int k = 0; k < 4; ++k) h[j][k] = fma2(h[j][k], w[k], v[k]);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) h[j][k] = add2(h[j][k], v[k]);
    }
    if (on) store_pairs(static_cast<TX*>(a.h) + t * d + c, h[j]);
    else zero8(h[j]);
  }
  if (a.pre_gamma == nullptr) return;
  const float rstd_h = centre();
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const int c = c0 + j * VSTEP;
    const bool on = c < d;
    load_param(on, a.pre_gamma + pc + j * VSTEP, v);
    load_param(on, a.pre_beta + pc + j * VSTEP, w);
#pragma unroll
    for (int k = 0; k < 4; ++k) h[j][k] = fma2(mul2(h[j][k], both(rstd_h)), v[k], w[k]);
    if (a.y_dtype == MTGR_F32) {
      if (on) store_pairs(static_cast<float*>(a.y) + t * d + c, h[j]);
    } else if (a.y_dtype == MTGR_BF16) {
      if (on) store_pairs(static_cast<__nv_bfloat16*>(a.y) + t * d + c, h[j]);
    } else if (on) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = unpair2(h[j][k]);
        m = max_nan(m, max_nan(fabsf(f.x), fabsf(f.y)));
      }
    }
  }
  if (a.y_dtype != MTGR_I8) return;
  const RowScale rs = row_scale(sums.max_bits(__float_as_uint(m)));
  if (tl == 0 && d > 0) a.y_scale[t] = rs.s;
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const int c = c0 + j * VSTEP;
    if (c < d) *reinterpret_cast<uint2*>(static_cast<int8_t*>(a.y) + t * d + c) = quant8(h[j], rs);
  }
}

template <typename TO, typename TX>
int launch_fwd_t(const BoundaryFwdArgs& a, cudaStream_t s) {
  const auto blocks = [&](int rows) { return (unsigned)(((int64_t)a.T + rows - 1) / rows); };
  if (a.d <= 64) boundary_fwd_kernel<TO, TX, 1, 8, 1><<<blocks(8), 64, 0, s>>>(a);
  else if (a.d <= 128) boundary_fwd_kernel<TO, TX, 1, 16, 1><<<blocks(4), 64, 0, s>>>(a);
  else if (a.d <= 256) boundary_fwd_kernel<TO, TX, 1, 32, 1><<<blocks(2), 64, 0, s>>>(a);
  else if (a.d <= 512) boundary_fwd_kernel<TO, TX, 1, 32, 2><<<blocks(2), 64, 0, s>>>(a);
  else if (a.d <= 1024) boundary_fwd_kernel<TO, TX, 2, 32, 2><<<a.T, 64, 0, s>>>(a);
  else if (a.d <= 2048) boundary_fwd_kernel<TO, TX, 4, 32, 2><<<a.T, 128, 0, s>>>(a);
  else if (a.d <= 4096) boundary_fwd_kernel<TO, TX, 8, 32, 2><<<a.T, 256, 0, s>>>(a);
  else boundary_fwd_kernel<TO, TX, 16, 32, 2><<<a.T, 512, 0, s>>>(a);
  return launch_status();
}

// --------------------------------------------------------------- backward --
enum { kPreGamma = 0, kPreBeta = 1, kScale = 2, kPostGamma = 3, kPostBeta = 4 };

// A row's inputs wait in shared memory: each thread copies its own eight values of
// every input one row ahead (cp.async; kAhead) and reads back only those, so no barrier
// is needed, and the registers hold the sums instead. Stage layout: per thread
// o, u (16 or 32 bytes), x, dh, dy; a thread's 16-byte pieces lie THREADS * 16
// bytes apart, so that a warp's accesses fall in different banks.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
template <typename T>
__device__ __forceinline__ void copy8(uint4* dst, int step, const T* src) {
#pragma unroll
  for (int i = 0; i < kPieces<T>; ++i)
    copy16((uint32_t)__cvta_generic_to_shared(dst + i * step), reinterpret_cast<const char*>(src) + 16 * i);
}
// plain loads: the compiler may move them ahead of the exchanges before them
template <typename T>
__device__ __forceinline__ void read8(const uint4* src, int step, f2 (&v)[4]) {
  const uint4 a = src[0];
  uint4 b = a;
  if constexpr (sizeof(T) == 4) b = src[step];
  to_pairs(a, b, v, T());
}
// Rows in flight beside the one computed. The largest teams' rows alone fill the
// shared memory: none ahead, and the parameters read from memory.
template <int WARPS>
constexpr int kAhead = WARPS == 16 ? 0 : 1;

// 16-byte pieces a thread keeps per vector of eight columns: its rows' inputs, and
// the parameters (post gamma and beta, scale, pre gamma) of the group at hand.
template <typename TO, typename TX>
constexpr int kRowPieces = 2 * kPieces<TO> + 2 * kPieces<TX> + 2;
template <int WARPS>
constexpr int kParamPieces = WARPS == 16 ? 0 : 8;

template <typename TO, typename TX, int WARPS, int VPL>
constexpr int bwd_thread_bytes() {
  return 16 * VPL * (kParamPieces<WARPS> + (kAhead<WARPS> + 1) * kRowPieces<TO, TX>);
}

// Blocks an SM holds at once, by registers: 12 warps of one vector a thread, 8 of two
// (16 of one, with spills, took 373 us against 249 at 200003 x 256).
constexpr int bwd_blocks(int warps, int vpl) {
  const int all = vpl == 1 ? 12 : 8, per = warps == 1 ? 4 : warps;
  return all / per > 0 ? all / per : 1;
}

// A team takes a contiguous run of rows (a user's segments are runs of one
// group, so the group seldom changes): LANES lanes of a warp (8 for d <= 64, 16 for
// d <= 128, 32 up to 512), four warps to a block; above, a block of WARPS warps. VPL vectors of eight columns a thread: two, so that a
// thread has two independent chains and a row few exchanges (at 200003 x 512: 573
// us with one vector and two warps a row). The parameter gradients gather in
// registers while the group stays the same; then they go to the team's own slots
// of the workspace (each thread its own columns: no atomics, and the same order of
// sums in every run).
template <typename TO, typename TX, int WARPS, int LANES, int VPL>
__global__ void __launch_bounds__(WARPS == 1 ? 128 : 32 * WARPS, bwd_blocks(WARPS, VPL))
    boundary_bwd_kernel(BoundaryBwdArgs a) {
  constexpr int AHEAD = kAhead<WARPS>, PP = kParamPieces<WARPS>;
  dependents_may_launch();
  extern __shared__ uint4 smem[];
  __shared__ float part[4 * WARPS];
  Sums<WARPS, LANES> sums{part};
  constexpr bool BLOCK = WARPS > 1;
  const int tl = BLOCK ? threadIdx.x : threadIdx.x % LANES;
  const int64_t ti = BLOCK ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * (128 / LANES) + threadIdx.x / LANES;
  if (LANES == 32 && ti >= a.teams) return;
  const int d = a.d;
  constexpr int VSTEP = 8 * LANES * WARPS;  // columns between a thread's vectors
  const int c0 = 8 * tl;
  bool on[VPL];
#pragma unroll
  for (int j = 0; j < VPL; ++j) on[j] = c0 + j * VSTEP < d;
  const int64_t t0 = ti * a.rows_per_team;
  const int rows = ti < a.teams ? (int)min((int64_t)a.rows_per_team, (int64_t)a.T - t0) : 0;
  // the warp's teams go through the loop together: one whose rows are done leaves its
  // sums, goes on with rows of zeros and keeps nothing of them (with eps = 0 their 1 / sigma
  // is infinite, and what they add NaN)
  const int most = LANES == 32 ? rows : (int)__reduce_max_sync(0xffffffffu, (unsigned)rows);
  const bool post = a.post_gamma != nullptr, pre = a.pre_gamma != nullptr, gate = a.gate != MTGR_GATE_NONE;
  const float inv_d = 1.0f / (float)d;
  float* slots = a.part + ti * a.G * kSlots * d + c0;
  // this thread's pieces lie `step` pieces apart (its neighbours' between them): the parameters', then the
  // stages', vector by vector
  constexpr int RP = kRowPieces<TO, TX>, PO = kPieces<TO>, PX = kPieces<TX>;
  constexpr int step = WARPS == 1 ? 128 : 32 * WARPS, stage = VPL * RP * step;
  uint4* params = smem + threadIdx.x;
  uint4* base = params + VPL * PP * step;

  f2 acc[kSlots][VPL][4];
#pragma unroll
  for (int i = 0; i < kSlots; ++i)
#pragma unroll
    for (int j = 0; j < VPL; ++j) zero8(acc[i][j]);
  uint32_t seen = 0u;
  int g_run = -1;
  bool range_bad = false;

  auto flush = [&]() {
    if (g_run < 0 || rows <= 0) return;  // a team past the last one has no slots
    float* p = slots + (int64_t)g_run * kSlots * d;
    const bool add = (seen >> g_run) & 1u;
#pragma unroll
    for (int i = 0; i < kSlots; ++i)
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        if (on[j]) {
          float* q = p + (int64_t)i * d + j * VSTEP;
          if (add) {
            f2 v[4];
            to_pairs(*reinterpret_cast<const uint4*>(q), *reinterpret_cast<const uint4*>(q + 4), v, 0.f);
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[i][j][k] = add2(acc[i][j][k], v[k]);
          }
          store_pairs(q, acc[i][j]);
        }
        zero8(acc[i][j]);
      }
    seen |= 1u << g_run;
  };
  // the group's parameters to this thread's pieces (0 past d)
  auto take_params = [&](int g) {
    if constexpr (PP == 0) return;
    const int64_t pc = (int64_t)g * d + c0;
    const float* src[4] = {a.post_gamma, a.post_beta, a.scale, a.pre_gamma};
#pragma unroll
    for (int j = 0; j < VPL; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint4 x = make_uint4(0u, 0u, 0u, 0u), y = x;
        if (on[j] && src[i] != nullptr) {
          x = *reinterpret_cast<const uint4*>(src[i] + pc + j * VSTEP);
          y = *reinterpret_cast<const uint4*>(src[i] + pc + j * VSTEP + 4);
        }
        uint4* to = params + (j * PP + 2 * i) * step;
        to[0] = x;
        to[step] = y;
      }
  };
  auto param = [&](int i, int j, f2 (&v)[4]) {
    if constexpr (PP == 0) {
      zero8(v);
      if (on[j]) {
        const float* src = i == 0 ? a.post_gamma : i == 1 ? a.post_beta : i == 2 ? a.scale : a.pre_gamma;
        src += (int64_t)g_run * d + c0 + j * VSTEP;
        to_pairs(*reinterpret_cast<const uint4*>(src), *reinterpret_cast<const uint4*>(src + 4), v, 0.f);
      }
    } else {
      read8<float>(params + (j * PP + 2 * i) * step, step, v);
    }
  };
  auto copy_row = [&](int r, int s) {
    if (r < rows) {
      const int64_t t = t0 + r;
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        if (!on[j]) continue;
        const int c = c0 + j * VSTEP;
        uint4* at = base + s * stage + j * RP * step;
        copy8(at, step, static_cast<const TO*>(a.o) + t * a.ld_o + c);
        if (gate) copy8(at + PO * step, step, static_cast<const TO*>(a.u) + t * a.ld_u + c);
        if (a.dh != nullptr) copy8(at + (2 * PO + PX) * step, step, static_cast<const TX*>(a.dh) + t * d + c);
        if (pre) {
          copy8(at + 2 * PO * step, step, static_cast<const TX*>(a.x) + t * d + c);
          if (a.dy_dtype == MTGR_F32)
            copy8(at + (2 * PO + 2 * PX) * step, step, static_cast<const float*>(a.dy) + t * d + c);
          else
            copy8(at + (2 * PO + 2 * PX) * step, step, static_cast<const __nv_bfloat16*>(a.dy) + t * d + c);
        }
      }
    } else if (LANES < 32) {
      for (int i = 0; i < VPL * RP; ++i) base[s * stage + i * step] = make_uint4(0u, 0u, 0u, 0u);
    }
    copy_commit();
  };
  // what is read past d is 0 throughout, so it adds nothing to a sum
#pragma unroll
  for (int j = 0; j < VPL; ++j)
    if (!on[j])
      for (int s = 0; s <= AHEAD; ++s)
        for (int i = 0; i < RP; ++i) base[s * stage + (j * RP + i) * step] = make_uint4(0u, 0u, 0u, 0u);

#pragma unroll
  for (int r = 0; r < AHEAD; ++r) copy_row(r, r);
  int g = rows > 0 ? clamp_group(a.gid, t0, a.G) : 0, s = 0;
  for (int r = 0; r < most; ++r) {
    const bool live = LANES == 32 || r < rows;
    copy_row(r + AHEAD, s == 0 ? AHEAD : s - 1);  // stage (s + AHEAD) mod (AHEAD + 1)
    const int g_next = r + 1 < rows ? clamp_group(a.gid, t0 + r + 1, a.G) : g;
    if (g != g_run || (LANES < 32 && r == rows)) {
      flush();
      g_run = g;
      take_params(g);
    }
    copy_wait<AHEAD>();
    const uint4* at = base + s * stage;
    const int64_t t = t0 + r;
    // n and p = n f again
    f2 oh[VPL][4], n[VPL][4], p[VPL][4], v[VPL][4], w[4];
    float rstd_o = 1.f;
#pragma unroll
    for (int j = 0; j < VPL; ++j) read8<TO>(at + j * RP * step, step, oh[j]);
    if (post) {
      f2 q = 0ull;
#pragma unroll
      for (int j = 0; j < VPL; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) q = add2(q, oh[j][k]);
      const f2 m = both(-sums(sum_of(q)) * inv_d);
      float sq = 0.f;
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        q = 0ull;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          oh[j][k] = add2(oh[j][k], m);
          q = fma2(oh[j][k], oh[j][k], q);
        }
        sq += on[j] ? sum_of(q) : 0.f;
      }
      rstd_o = rsqrtf(sums(sq) * inv_d + a.eps);
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        param(0, j, v[j]);
        param(1, j, w);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          oh[j][k] = mul2(oh[j][k], both(rstd_o));
          n[j][k] = fma2(oh[j][k], v[j][k], w[k]);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < VPL; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) n[j][k] = oh[j][k];
    }
    f2 f[VPL][4], sc[VPL][4];
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      if (gate) {
        read8<TO>(at + (j * RP + PO) * step, step, f[j]);
        if (a.gate == MTGR_GATE_SILU) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 u = unpair2(f[j][k]);
            f[j][k] = pair2(silu_f32(u.x), silu_f32(u.y));
          }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) p[j][k] = mul2(n[j][k], f[j][k]);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          f[j][k] = both(1.f);
          p[j][k] = n[j][k];
        }
      }
      if (a.scale != nullptr) {
        param(2, j, sc[j]);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) sc[j][k] = both(1.f);
      }
    }
    // H: the gradient at h
    f2 H[VPL][4];
    if (pre) {
      f2 hh[VPL][4], m = 0ull;
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        read8<TX>(at + (j * RP + 2 * PO) * step, step, hh[j]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          hh[j][k] = fma2(p[j][k], sc[j][k], hh[j][k]);
          m = add2(m, hh[j][k]);
        }
      }
      const f2 mean = both(-sums(sum_of(m)) * inv_d);
      float sq = 0.f;
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        f2 q = 0ull;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          hh[j][k] = add2(hh[j][k], mean);
          q = fma2(hh[j][k], hh[j][k], q);
        }
        sq += on[j] ? sum_of(q) : 0.f;
      }
      const float rstd_h = rsqrtf(sums(sq) * inv_d + a.eps);
      f2 m0 = 0ull, m1 = 0ull;
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        const uint4* from = at + (j * RP + 2 * PO + 2 * PX) * step;
        if (a.dy_dtype == MTGR_F32) read8<float>(from, step, v[j]);
        else read8<__nv_bfloat16>(from, step, v[j]);
        param(3, j, w);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          hh[j][k] = mul2(hh[j][k], both(rstd_h));
          acc[kPreGamma][j][k] = fma2(v[j][k], hh[j][k], acc[kPreGamma][j][k]);
          acc[kPreBeta][j][k] = add2(acc[kPreBeta][j][k], v[j][k]);
          v[j][k] = mul2(v[j][k], w[k]);
          m0 = add2(m0, v[j][k]);
          m1 = fma2(v[j][k], hh[j][k], m1);
        }
      }
      const float2 ms = sums(sum_of(m0), sum_of(m1));
      const f2 c0n = both(-ms.x * inv_d), c1n = both(-ms.y * inv_d);
#pragma unroll
      for (int j = 0; j < VPL; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) H[j][k] = mul2(both(rstd_h), fma2(hh[j][k], c1n, add2(v[j][k], c0n)));
    } else {
#pragma unroll
      for (int j = 0; j < VPL; ++j) zero8(H[j]);
    }
    f2 m0 = 0ull, m1 = 0ull;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const int c = c0 + j * VSTEP;
      if (a.dh != nullptr) {
        read8<TX>(at + (j * RP + 2 * PO + PX) * step, step, v[j]);
#pragma unroll
        for (int k = 0; k < 4; ++k) H[j][k] = add2(H[j][k], v[j][k]);
      }
      if (on[j] && live) store_pairs(static_cast<TX*>(a.dx) + t * d + c, H[j]);
      // sc becomes the gradient at p
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        acc[kScale][j][k] = fma2(H[j][k], p[j][k], acc[kScale][j][k]);
        sc[j][k] = mul2(H[j][k], sc[j][k]);
      }
      if (gate) {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[j][k] = mul2(sc[j][k], n[j][k]);
        if (a.gate == MTGR_GATE_SILU) {
          f2 u[4];
          read8<TO>(at + (j * RP + PO) * step, step, u);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 x = unpair2(u[k]), y = unpair2(f[j][k]);
            const float s0 = sigmoid_f32(x.x), s1 = sigmoid_f32(x.y);
            // sigmoid(u) (1 + u (1 - sigmoid(u)))
            v[j][k] = mul2(v[j][k], pair2(fmaf(y.x, 1.0f - s0, s0), fmaf(y.y, 1.0f - s1, s1)));
          }
        }
        if (on[j] && live) {
          store_pairs(static_cast<TO*>(a.du) + t * a.ld_du + c, v[j]);
          if (sizeof(TO) == 2 && a.o_dtype == MTGR_F16) range_bad |= beyond_f16(v[j]);
        }
      }
      if (post) param(0, j, w);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const f2 dn = mul2(sc[j][k], f[j][k]);
        acc[kPostGamma][j][k] = fma2(dn, oh[j][k], acc[kPostGamma][j][k]);
        acc[kPostBeta][j][k] = add2(acc[kPostBeta][j][k], dn);
        v[j][k] = dn;
        if (post) {
          v[j][k] = mul2(dn, w[k]);
          m0 = add2(m0, v[j][k]);
          m1 = fma2(v[j][k], oh[j][k], m1);
        }
      }
    }
    if (post) {
      const float2 ms = sums(sum_of(m0), sum_of(m1));
      const f2 c0n = both(-ms.x * inv_d), c1n = both(-ms.y * inv_d);
#pragma unroll
      for (int j = 0; j < VPL; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) v[j][k] = mul2(both(rstd_o), fma2(oh[j][k], c1n, add2(v[j][k], c0n)));
    }
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      if (on[j] && live) {
        store_pairs(static_cast<TO*>(a.d_o) + t * a.ld_do + c0 + j * VSTEP, v[j]);
        if (sizeof(TO) == 2 && a.o_dtype == MTGR_F16) range_bad |= beyond_f16(v[j]);
      }
    }
    g = g_next;
    s = s == AHEAD ? 0 : s + 1;
  }
  if (rows == most) flush();  // the others left theirs when their rows were done
  if (tl == 0 && ti < a.teams) a.seen[ti] = seen;
  if (range_bad) set_status(a.status, MTGR_ERR_RANGE);
}

// The parameter gradients: each of the G * 5 * d columns summed over the teams
// that saw its group, in fp64 and a fixed order: a block per 32 columns, four a
// thread, its 64 groups of eight threads over the teams.
__global__ void __launch_bounds__(512) boundary_bwd_reduce_kernel(BoundaryBwdArgs a) {
  __shared__ double red[64][8][4];
  const int cl = threadIdx.x & 7, part = threadIdx.x >> 3;
  const int64_t n = (int64_t)a.G * kSlots * a.d;
  const int64_t c = ((int64_t)blockIdx.x * 8 + cl) * 4;  // d % 8 == 0: one slot and group per 4 columns
  const int gs = c < n ? (int)(c / a.d) : 0;
  const int g = gs / kSlots, slot = gs % kSlots;
  float* out = slot == kPreGamma    ? a.g_pre_gamma
               : slot == kPreBeta   ? a.g_pre_beta
               : slot == kScale     ? a.g_scale
               : slot == kPostGamma ? a.g_post_gamma
                                    : a.g_post_beta;
  dependent_wait();
  double s[4] = {0.0, 0.0, 0.0, 0.0};
  if (c < n && out != nullptr) {
#pragma unroll 4
    for (int i = part; i < a.teams; i += 64) {
      if ((a.seen[i] >> g) & 1u) {
        const float4 v = *reinterpret_cast<const float4*>(a.part + i * n + c);
        s[0] += v.x; s[1] += v.y; s[2] += v.z; s[3] += v.w;
      }
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) red[part][cl][k] = s[k];
  __syncthreads();
  // 32 columns, 16 threads each over four partials, then across the 16
  const int col = threadIdx.x >> 4, w = threadIdx.x & 15;
  double t = 0.0;
#pragma unroll
  for (int k = 0; k < 4; ++k) t += red[4 * w + k][col >> 2][col & 3];
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  const int64_t cc = (int64_t)blockIdx.x * 32 + col;
  if (w != 0 || cc >= n) return;
  const int gs2 = (int)(cc / a.d), slot2 = gs2 % kSlots;
  float* to = slot2 == kPreGamma    ? a.g_pre_gamma
              : slot2 == kPreBeta   ? a.g_pre_beta
              : slot2 == kScale     ? a.g_scale
              : slot2 == kPostGamma ? a.g_post_gamma
                                    : a.g_post_beta;
  if (to != nullptr) to[(int64_t)(gs2 / kSlots) * a.d + (cc - (int64_t)gs2 * a.d)] = (float)t;
}

// Warps of a row's team and vectors a thread.
inline int bwd_warps(int d) { return d <= 512 ? 1 : (d <= 1024 ? 2 : (d <= 2048 ? 4 : (d <= 4096 ? 8 : 16))); }
inline int bwd_vpl(int d) { return d <= 256 ? 1 : 2; }
inline int bwd_lanes(int d) { return d <= 64 ? 8 : (d <= 128 ? 16 : 32); }

// Most teams that any types of this width have resident at once.
int64_t bwd_resident(int32_t d) {
  const int warps = bwd_warps(d);
  return (int64_t)device_sm_count() * bwd_blocks(warps, bwd_vpl(d)) * (warps == 1 ? 128 / bwd_lanes(d) : 1);
}

template <typename TO, typename TX, int WARPS, int LANES, int VPL>
int launch_bwd_w(BoundaryBwdArgs& a, cudaStream_t s) {
  constexpr int threads = WARPS == 1 ? 128 : 32 * WARPS;
  constexpr int bytes = threads * bwd_thread_bytes<TO, TX, WARPS, VPL>();
  // blocks an SM holds at once: by registers, and by shared memory (228 KB, 1 KB of
  // it per block for the system); a team that waited for another to end would
  // double the time
  constexpr int by_smem = 228 * 1024 / (bytes + 16 * WARPS + 1024);
  static_assert(by_smem >= 1, "shared memory of a block");
  constexpr int by_regs = bwd_blocks(WARPS, VPL);
  constexpr int blocks = by_regs < by_smem ? by_regs : by_smem;
  constexpr int per_block = WARPS == 1 ? 128 / LANES : 1;
  a.teams = bwd_teams(a.T, a.d, a.G, (int64_t)device_sm_count() * blocks * per_block);
  a.rows_per_team = rows_per_team(a.T, a.teams);
  auto kern = boundary_bwd_kernel<TO, TX, WARPS, LANES, VPL>;
  if (bytes > 40 * 1024 &&  // 48 KB without asking, some of it static
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
    return MTGR_ERR_CUDA;
  kern<<<(a.teams + per_block - 1) / per_block, threads, bytes, s>>>(a);
  return launch_status();
}

template <typename TO, typename TX>
int launch_bwd_t(BoundaryBwdArgs& a, cudaStream_t s) {
  if (a.T > 0) {
    int rc = MTGR_OK;
    if (a.d <= 64) rc = launch_bwd_w<TO, TX, 1, 8, 1>(a, s);
    else if (a.d <= 128) rc = launch_bwd_w<TO, TX, 1, 16, 1>(a, s);
    else if (a.d <= 256) rc = launch_bwd_w<TO, TX, 1, 32, 1>(a, s);
    else if (a.d <= 512) rc = launch_bwd_w<TO, TX, 1, 32, 2>(a, s);
    else if (a.d <= 1024) rc = launch_bwd_w<TO, TX, 2, 32, 2>(a, s);
    else if (a.d <= 2048) rc = launch_bwd_w<TO, TX, 4, 32, 2>(a, s);
    else if (a.d <= 4096) rc = launch_bwd_w<TO, TX, 8, 32, 2>(a, s);
    else rc = launch_bwd_w<TO, TX, 16, 32, 2>(a, s);
    if (rc != MTGR_OK) return rc;
  }
  const int64_t n = (int64_t)a.G * kSlots * a.d;
  return launch_dependent(boundary_bwd_reduce_kernel, (unsigned)((n + 31) / 32), 512, 0, s, a);
}

}  // namespace

size_t boundary_bwd_ws_bytes(int32_t T, int32_t d, int32_t G) {
  const size_t teams = (size_t)bwd_teams(T, d, G, bwd_resident(d));
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
  a.teams = a.rows_per_team = 0;  // set with the form
  a.seen = static_cast<uint32_t*>(ws);
  a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) +
                                    align_up((size_t)bwd_teams(a.T, a.d, a.G, bwd_resident(a.d)) * 4, 256));
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
