// The global 2-norm over many gradient tensors, the loss scale taken out, and
// clipping (the block's gradients, of a loss that f16 training scales):
//   norm = inv_scale sqrt(sum g^2),  c = inv_scale min(1, max_norm / (norm + 1e-6)),  out = g c
// Small sets: one kernel that keeps what it read (below). Others: two kernels over
// all tensors, the first sums squares (each gradient read once), the second scales
// (read again, from L2 where the set fits, and written). The tensors travel as a
// table in the kernel's parameters, so nothing is copied to the device ahead. Large
// sets are bound by HBM, small ones by the launch and the meeting of the blocks.
//
// Sums: squares of eight values in fp32, over those in fp64 (eight positive terms are off by
// eight roundings of 2^-24 at most, which the root halves; fp64 throughout would take
// eight conversions for one); where the eight leave fp32's range (values beyond 1e18 or all
// below 1e-18), they are squared in fp64. Blocks write their sums to the workspace, and they are added in a
// fixed order: no atomics on values, the same norm in every run.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "ops.h"
#include "rowvec.cuh"

namespace mtgr {

namespace {

// Tensors per launch: a launch costs more the more it carries (2.9 against 0.5 KB of
// parameters), so small sets go in a small table.
constexpr int kTable = 96, kSmallTable = 16;
constexpr int64_t kChunk = 16384;     // elements a block takes at a time

__device__ __forceinline__ uint64_t globaltimer_now() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

template <int N>
struct Table {
  const void* g[N];
  void* out[N];
  int64_t n[N];
  int32_t chunk0[N + 1];  // first chunk of each tensor
  uint8_t dtype[N];       // in | out << 4
  int32_t count;
};

// The tensor of a chunk: the last one whose first chunk is not behind it. All
// lanes look at once, by generic loads: a search by halves costs seven misses of the
// constant cache in a row, most of a small set's time.
template <int N>
__device__ __forceinline__ int find_tensor(const Table<N>& t, int chunk) {
  constexpr int R = (N + 31) / 32;
  const int lane = threadIdx.x & 31;
  int n = 0, first[R];
#pragma unroll
  for (int i = 0; i < R; ++i)
    asm volatile("ld.s32 %0, [%1];" : "=r"(first[i]) : "l"(&t.chunk0[min(lane + 32 * i, N)]));
#pragma unroll
  for (int i = 0; i < R; ++i)
    n += __popc(__ballot_sync(0xffffffffu, lane + 32 * i < t.count && first[i] <= chunk));
  return n - 1;
}

__device__ __forceinline__ double square8(const float (&v)[8]) {
  float s = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) s = fmaf(v[e], v[e], s);
  if (s > 1e-30f && s < 1e36f) return (double)s;  // no square that matters was lost or overflowed
  double q = 0.0;
#pragma unroll
  for (int e = 0; e < 8; ++e) q = fma((double)v[e], (double)v[e], q);
  return q;
}

template <typename T>
__device__ __forceinline__ float to_float(T v) { return static_cast<float>(v); }

// One chunk [e0, e1) of a tensor: whole vectors of eight where the address is
// 16-byte aligned, single elements before and after.
template <typename T>
__device__ __forceinline__ double sum_chunk(const void* gv, int64_t e0, int64_t e1) {
  const T* g = static_cast<const T*>(gv);
  const uintptr_t addr = reinterpret_cast<uintptr_t>(g + e0);
  const int64_t head = min(e1, e0 + (int64_t)(((16 - (addr & 15)) & 15) / sizeof(T)));
  const int64_t nv = (e1 - head) / 8;
  double s = 0.0;
  const int64_t singles = (head - e0) + (e1 - head - 8 * nv);
  for (int64_t i = threadIdx.x; i < singles; i += blockDim.x) {
    const double v = to_float(g[i < head - e0 ? e0 + i : head + 8 * nv + (i - (head - e0))]);
    s = fma(v, v, s);
  }
#pragma unroll 4
  for (int64_t i = threadIdx.x; i < nv; i += blockDim.x) {
    Vec8<T> r;
    r.load(g + head + 8 * i);
    float v[8];
    r.unpack(v);
    s += square8(v);
  }
  return s;
}

__device__ __forceinline__ double block_sum(double s) {
  __shared__ double red[32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
  __syncthreads();
  s = (threadIdx.x & 31) < (blockDim.x >> 5) ? red[threadIdx.x & 31] : 0.0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

template <int N>
__global__ void __launch_bounds__(256) grad_sum_kernel(const __grid_constant__ Table<N> t, double* part) {
  double s = 0.0;
  const int chunks = t.chunk0[t.count];
  for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int i = find_tensor(t, c);
    const int64_t e0 = (int64_t)(c - t.chunk0[i]) * kChunk;
    const int64_t e1 = min(t.n[i], e0 + kChunk);
    const int in = t.dtype[i] & 15;
    if (in == MTGR_F32) s += sum_chunk<float>(t.g[i], e0, e1);
    else if (in == MTGR_BF16) s += sum_chunk<__nv_bfloat16>(t.g[i], e0, e1);
    else s += sum_chunk<__half>(t.g[i], e0, e1);
  }
  s = block_sum(s);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }

// The factor of the clip, c 2^e; e = 0 where c is one of fp32's normal numbers. Below them
// (an exploded step: norm 1e38 to 1) c would have lost bits, or be 0, while its products
// with such gradients are ordinary numbers.
struct Factor {
  float c;
  int32_t e;
};
__device__ __forceinline__ Factor clip_factor(double norm, float max_norm, float inv_scale) {
  const double ratio = (double)max_norm / (norm + 1e-6);
  Factor f{inv_scale * fminf(1.0f, (float)ratio), 0};
  if (f.c < 1.17549435e-38f) f.c = (float)frexp((double)inv_scale * fmin(1.0, ratio), &f.e);
  return f;
}

template <typename T, typename O>
__device__ __forceinline__ void scale_chunk(const void* gv, void* ov, int64_t e0, int64_t e1, float c, int32_t exp2) {
  const T* g = static_cast<const T*>(gv);
  O* o = static_cast<O*>(ov);
  const uintptr_t ga = reinterpret_cast<uintptr_t>(g + e0), oa = reinterpret_cast<uintptr_t>(o + e0);
  int64_t head = min(e1, e0 + (int64_t)(((16 - (ga & 15)) & 15) / sizeof(T)));
  // vectors only where both sides are aligned from the same element on, and the factor is an
  // ordinary one
  const bool vec = ((oa + (uintptr_t)(head - e0) * sizeof(O)) & 15) == 0;
  if (!vec || exp2 != 0) head = e1;
  const int64_t nv = (e1 - head) / 8;
  const int64_t singles = (head - e0) + (e1 - head - 8 * nv);
  for (int64_t i = threadIdx.x; i < singles; i += blockDim.x) {
    const int64_t e = i < head - e0 ? e0 + i : head + 8 * nv + (i - (head - e0));
    const float v = to_float(g[e]) * c;
    o[e] = from_float<O>(exp2 == 0 ? v : ldexpf(v, exp2));
  }
#pragma unroll 4
  for (int64_t i = threadIdx.x; i < nv; i += blockDim.x) {
    Vec8<T> r;
    r.load(g + head + 8 * i);
    float v[8];
    r.unpack(v);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= c;
    store8(o + head + 8 * i, v);
  }
}

// parts: the sums of all launches of the first kernel. scale == 0: the norm only.
template <int N>
__global__ void __launch_bounds__(256) grad_scale_kernel(const __grid_constant__ Table<N> t, const double* part,
                                                         int32_t parts, float max_norm, float inv_scale,
                                                         int32_t scale, float* norm_out, int32_t* status) {
  double s = 0.0;
  for (int i = threadIdx.x; i < parts; i += blockDim.x) s += part[i];
  s = block_sum(s);
  const double norm = sqrt(s) * (double)inv_scale;
  const bool finite = isfinite((float)norm);
  if (blockIdx.x == 0 && threadIdx.x == 0 && norm_out != nullptr) {
    *norm_out = (float)norm;
    if (!finite) set_status(status, MTGR_ERR_RANGE);
  }
  if (scale == 0 || !finite) return;
  const Factor f = clip_factor(norm, max_norm, inv_scale);
  const int chunks = t.chunk0[t.count];
  // last chunks first: they are the ones L2 still holds
  for (int k = chunks - 1 - (int)blockIdx.x; k >= 0; k -= gridDim.x) {
    const int i = find_tensor(t, k);
    const int64_t e0 = (int64_t)(k - t.chunk0[i]) * kChunk;
    const int64_t e1 = min(t.n[i], e0 + kChunk);
    if (f.c == 1.0f && f.e == 0 && t.g[i] == t.out[i]) continue;  // nothing to change in place
    switch (t.dtype[i]) {
      case MTGR_F32 | MTGR_F32 << 4: scale_chunk<float, float>(t.g[i], t.out[i], e0, e1, f.c, f.e); break;
      case MTGR_BF16 | MTGR_BF16 << 4: scale_chunk<__nv_bfloat16, __nv_bfloat16>(t.g[i], t.out[i], e0, e1, f.c, f.e); break;
      case MTGR_F16 | MTGR_F16 << 4: scale_chunk<__half, __half>(t.g[i], t.out[i], e0, e1, f.c, f.e); break;
      case MTGR_BF16 | MTGR_F32 << 4: scale_chunk<__nv_bfloat16, float>(t.g[i], t.out[i], e0, e1, f.c, f.e); break;
      default: scale_chunk<__half, float>(t.g[i], t.out[i], e0, e1, f.c, f.e); break;
    }
  }
}

// -------------------------------------------------- small sets, one kernel --
// A set whose values fit the registers of blocks that all run at once is read once:
// every thread keeps up to kHeld vectors of eight, the blocks meet (a cooperative
// launch, so none waits for one that cannot run), and each scales what it holds.
// The two launches of the other form took 18.4 us a pass at a block of width 512 (3.1 M
// values, cold), this 10.4; in a graph and from L2 4.8 M values take 12.5 and 11.8 us,
// 40,000 values 8.4 and 5.1. The loads of a thread's vectors are all on their way
// before the first is squared. A set behind the border runs at the memory's rate
// either way.
constexpr int kHeld = 4, kHeldThreads = 512, kHeldBlocks = 2;  // blocks an SM
constexpr int64_t kHeldChunk = kHeldThreads * 8;

struct Meet {  // in the workspace, zero between calls
  uint32_t arrived, left;
};

template <typename T>
__device__ __forceinline__ void load_some(const void* gv, int64_t at, int64_t n, float (&v)[8]) {
  const T* g = static_cast<const T*>(gv) + at;
  if (at + 8 <= n && (reinterpret_cast<uintptr_t>(g) & 15) == 0) {
    Vec8<T> r;
    r.load(g);
    r.unpack(v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = at + e < n ? to_float(g[e]) : 0.f;
  }
}
template <typename O>
__device__ __forceinline__ void store_some(void* ov, int64_t at, int64_t n, const float (&v)[8]) {
  O* o = static_cast<O*>(ov) + at;
  if (at + 8 <= n && (reinterpret_cast<uintptr_t>(o) & 15) == 0) {
    store8(o, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (at + e < n) o[e] = from_float<O>(v[e]);
  }
}

template <int N>
__global__ void __launch_bounds__(kHeldThreads, kHeldBlocks)
    grad_clip_held_kernel(const __grid_constant__ Table<N> t, Meet* meet, double* part, float max_norm,
                          float inv_scale, int32_t scale, float* norm_out, int32_t* status) {
  __shared__ int32_t met;
  float v[kHeld][8];
  int which[kHeld];
  const int chunks = t.chunk0[t.count];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int c = blockIdx.x + i * (int)gridDim.x;
    which[i] = c < chunks ? find_tensor(t, c) : -1;
  }
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int k = which[i];
    if (k < 0) continue;
    const int64_t at = (int64_t)(blockIdx.x + i * (int)gridDim.x - t.chunk0[k]) * kHeldChunk + 8 * threadIdx.x;
    const int in = t.dtype[k] & 15;
    if (in == MTGR_F32) load_some<float>(t.g[k], at, t.n[k], v[i]);
    else if (in == MTGR_BF16) load_some<__nv_bfloat16>(t.g[k], at, t.n[k], v[i]);
    else load_some<__half>(t.g[k], at, t.n[k], v[i]);
  }
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (which[i] >= 0) s += square8(v[i]);
  s = block_sum(s);
  if (threadIdx.x == 0) {
    part[blockIdx.x] = s;
    __threadfence();
    atomicAdd(&meet->arrived, 1u);
    const uint64_t t0 = globaltimer_now();
    int32_t ok = 1;
    for (int i = 1;; ++i) {
      uint32_t a;
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(a) : "l"(&meet->arrived) : "memory");
      if (a == gridDim.x) break;
      if ((i & 63) == 0 && globaltimer_now() - t0 > kWaitLimitNs) {
        ok = 0;
        break;
      }
    }
    met = ok;
    // the last block to pass leaves the words as it found them
    if (atomicAdd(&meet->left, 1u) == gridDim.x - 1) meet->arrived = meet->left = 0u;
    if (!ok) set_status(status, MTGR_ERR_TIMEOUT);
  }
  __syncthreads();
  if (!met) return;
  s = 0.0;
  for (int i = threadIdx.x; i < (int)gridDim.x; i += kHeldThreads) s += load_written(part + i);
  s = block_sum(s);
  const double norm = sqrt(s) * (double)inv_scale;
  const bool finite = isfinite((float)norm);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *norm_out = (float)norm;
    if (!finite) set_status(status, MTGR_ERR_RANGE);
  }
  if (scale == 0 || !finite) return;
  const Factor f = clip_factor(norm, max_norm, inv_scale);
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int k = which[i];
    if (k < 0 || (f.c == 1.0f && f.e == 0 && t.g[k] == t.out[k])) continue;
    const int64_t at = (int64_t)(blockIdx.x + i * (int)gridDim.x - t.chunk0[k]) * kHeldChunk + 8 * threadIdx.x;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[i][e] *= f.c;
    if (f.e != 0) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = ldexpf(v[i][e], f.e);
    }
    const int out = t.dtype[k] >> 4;
    if (out == MTGR_F32) store_some<float>(t.out[k], at, t.n[k], v[i]);
    else if (out == MTGR_BF16) store_some<__nv_bfloat16>(t.out[k], at, t.n[k], v[i]);
    else store_some<__half>(t.out[k], at, t.n[k], v[i]);
  }
}

// Blocks of a launch over `chunks` chunks.
int grid_of(int64_t chunks) {
  const int64_t most = (int64_t)device_sm_count() * 4;
  return (int)(chunks < 1 ? 1 : (chunks < most ? chunks : most));
}

int64_t chunks_of(int64_t n, int64_t chunk = kChunk) { return (n + chunk - 1) / chunk; }

// Chunks of a set for the one-kernel form; 0 if it does not fit.
int64_t held_chunks(const mtgr_grad_tensor* g, int32_t n) {
  if (n > kTable) return 0;
  const int64_t most = (int64_t)device_sm_count() * kHeldBlocks * kHeld;
  int64_t c = 0;
  for (int32_t i = 0; i < n && c <= most; ++i) c += chunks_of(g[i].n, kHeldChunk);
  return c <= most ? c : 0;
}

// Tensors [first, last) of one launch as a table; empty tensors take no chunk.
template <int N>
void fill(Table<N>& t, const mtgr_grad_tensor* g, int first, int last, int64_t chunk = kChunk) {
  int64_t c = 0;
  for (int i = first; i < last; ++i) {
    t.g[i - first] = g[i].g;
    t.out[i - first] = g[i].out;
    t.n[i - first] = g[i].n;
    t.dtype[i - first] = (uint8_t)(g[i].dtype | g[i].out_dtype << 4);
    t.chunk0[i - first] = (int32_t)c;
    c += chunks_of(g[i].n, chunk);
  }
  t.count = last - first;
  t.chunk0[t.count] = (int32_t)c;
}

template <int N>
int launch_n(const mtgr_grad_tensor* g, int32_t n, float max_norm, float inv_scale, float* norm,
                     void* ws, int32_t* status, cudaStream_t s) {
  Meet* meet = static_cast<Meet*>(ws);
  double* part = reinterpret_cast<double*>(static_cast<uint8_t*>(ws) + 256);
  Table<N> t;
  t.count = 0;
  t.chunk0[0] = 0;
  int32_t parts = 0;
  bool scale = false;
  if (const int64_t chunks = held_chunks(g, n); chunks > 0) {
    fill(t, g, 0, n, kHeldChunk);
    for (int k = 0; k < t.count; ++k) scale = scale || (t.n[k] > 0 && t.out[k] != nullptr);
    const int64_t most = (int64_t)device_sm_count() * kHeldBlocks;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(chunks < most ? chunks : most));
    cfg.blockDim = dim3(kHeldThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, grad_clip_held_kernel<N>, t, meet, part, max_norm, inv_scale,
                       (int32_t)(scale ? 1 : 0), norm, status);
    return launch_status();
  }
  for (int32_t i = 0; i < n; i += N) {
    fill(t, g, i, n < i + N ? n : i + N);
    for (int k = 0; k < t.count; ++k) scale = scale || (t.n[k] > 0 && t.out[k] != nullptr);
    const int grid = grid_of(t.chunk0[t.count]);
    grad_sum_kernel<N><<<grid, 256, 0, s>>>(t, part + parts);
    const int rc = launch_status();
    if (rc != MTGR_OK) return rc;
    parts += grid;
  }
  // the last table first, for what L2 holds; the norm is written once
  const int32_t last = n > 0 ? (n - 1) / N * N : 0;
  for (int32_t i = last; i >= 0; i -= N) {
    if (n > N) fill(t, g, i, n < i + N ? n : i + N);
    const int grid = scale ? grid_of(t.chunk0[t.count]) : 1;
    // (an early launch of this kernel beside the first one measured 250 against 213
    // us on 101 M fp32 values)
    grad_scale_kernel<N><<<grid, 256, 0, s>>>(t, part, parts, max_norm, inv_scale, scale ? 1 : 0,
                                          i == last ? norm : nullptr, status);
    const int rc = launch_status();
    if (rc != MTGR_OK) return rc;
    if (!scale) break;
  }
  return MTGR_OK;
}

}  // namespace

// The first kernel's blocks over all launches, 8 bytes each.
size_t grad_clip_ws_bytes(const mtgr_grad_tensor* g, int32_t n) {
  size_t parts = 0;
  for (int32_t i = 0; i < n; i += kTable) {
    int64_t c = 0;
    for (int32_t k = i; k < n && k < i + kTable; ++k) c += chunks_of(g[k].n);
    parts += (size_t)grid_of(c);
  }
  if (held_chunks(g, n) > 0) parts = (size_t)device_sm_count() * kHeldBlocks;
  return 256 + align_up(parts * 8, 256);
}

// Kernels of a call, for the timer.
int grad_clip_launches(const mtgr_grad_tensor* g, int32_t n) {
  if (held_chunks(g, n) > 0) return 1;
  const int tables = (n + kTable - 1) / kTable;
  for (int32_t i = 0; i < n; ++i)
    if (g[i].n > 0 && g[i].out != nullptr) return 2 * tables;
  return tables + 1;
}

int launch_grad_clip(const mtgr_grad_tensor* g, int32_t n, float max_norm, float inv_scale, float* norm,
                     void* ws, int32_t* status, cudaStream_t s) {
  return n <= kSmallTable ? launch_n<kSmallTable>(g, n, max_norm, inv_scale, norm, ws, status, s)
                          : launch_n<kTable>(g, n, max_norm, inv_scale, norm, ws, status, s);
}

}  // namespace mtgr
