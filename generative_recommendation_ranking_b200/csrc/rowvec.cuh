// Row vectors of eight elements for the row kernels (one row of [rows][d] per
// team of threads): 16- or 32-byte loads and stores of fp32, bf16 and f16, maxima over
// a team, and the quantisation of a row to signed bytes.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "common.cuh"

namespace mtgr {

// Eight consecutive elements as loaded, so that a thread's share of a row costs
// as few registers as its bytes.
template <typename T>
struct Vec8;

template <>
struct Vec8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void pairs(uint64_t (&v)[4]) const;
  __device__ __forceinline__ void unpack(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};

template <>
struct Vec8<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void pairs(uint64_t (&v)[4]) const;
  __device__ __forceinline__ void unpack(float (&v)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = __uint_as_float(w[k] << 16);
      v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
  }
};

template <>
struct Vec8<__half> {
  uint4 a;
  __device__ __forceinline__ void load(const __half* p) { a = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void pairs(uint64_t (&v)[4]) const;
  __device__ __forceinline__ void unpack(float (&v)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
      v[2 * k] = f.x;
      v[2 * k + 1] = f.y;
    }
  }
};

__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
    w[k] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(__half* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const __half2 h = __floats2half2_rn(v[2 * k], v[2 * k + 1]);
    w[k] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// ----------------------------------------------------------- packed pairs --
// Two fp32 values in one 64-bit register pair: sm_100 adds, multiplies and
// multiply-adds pairs in one instruction. Eight values are four pairs.
using f2 = uint64_t;
__device__ __forceinline__ f2 pair2(float lo, float hi) {
  f2 d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ float2 unpair2(f2 v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
__device__ __forceinline__ f2 both(float v) { return pair2(v, v); }
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ float sum_of(f2 a) {
  const float2 f = unpair2(a);
  return f.x + f.y;
}

// Eight elements as loaded (one or two 16-byte words) to four pairs.
__device__ __forceinline__ void to_pairs(const uint4& a, const uint4& b, f2 (&v)[4], float) {
  v[0] = pair2(__uint_as_float(a.x), __uint_as_float(a.y));
  v[1] = pair2(__uint_as_float(a.z), __uint_as_float(a.w));
  v[2] = pair2(__uint_as_float(b.x), __uint_as_float(b.y));
  v[3] = pair2(__uint_as_float(b.z), __uint_as_float(b.w));
}
__device__ __forceinline__ void to_pairs(const uint4& a, const uint4&, f2 (&v)[4], __nv_bfloat16) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = pair2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u));
}
__device__ __forceinline__ void to_pairs(const uint4& a, const uint4&, f2 (&v)[4], __half) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
    v[k] = pair2(f.x, f.y);
  }
}
__device__ __forceinline__ void Vec8<float>::pairs(uint64_t (&v)[4]) const {
  v[0] = pair2(a.x, a.y);
  v[1] = pair2(a.z, a.w);
  v[2] = pair2(b.x, b.y);
  v[3] = pair2(b.z, b.w);
}
__device__ __forceinline__ void Vec8<__nv_bfloat16>::pairs(uint64_t (&v)[4]) const {
  to_pairs(a, a, v, __nv_bfloat16());
}
__device__ __forceinline__ void Vec8<__half>::pairs(uint64_t (&v)[4]) const { to_pairs(a, a, v, __half()); }

template <typename T>
__device__ __forceinline__ void store_pairs(T* p, const f2 (&v)[4]) {
  float o[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f = unpair2(v[k]);
    o[2 * k] = f.x;
    o[2 * k + 1] = f.y;
  }
  store8(p, o);
}

// ------------------------------------------------------------------ teams --
// Maximum of non-negative values by their bits over a row's threads: one warp, or a
// whole block, whose warps meet in shared memory (part: 32 words). A NaN is above every
// number and an infinity, so it is not lost. Every thread gets the result.
template <bool BLOCK>
__device__ __forceinline__ uint32_t team_max_bits(uint32_t a, uint32_t* part) {
  a = __reduce_max_sync(0xffffffffu, a);
  if constexpr (BLOCK) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    if (lane == 0) part[warp] = a;
    __syncthreads();
    a = __reduce_max_sync(0xffffffffu, lane < nw ? part[lane] : 0u);
  }
  return a;
}

// -------------------------------------------------- rows in signed 8 bits --
// A row's scale s = max(max |v|, 2^-100) * (1 / 127), 1 / 127 rounded to fp32, and
// its values q = v / s rounded to the nearest integer, ties to even. 2^-100 keeps s and 1 / s normal numbers
// for a row of zeros or of the smallest values, whose q are then 0. A row with
// an infinity or a NaN gets s = NaN and q = 0, so that what reads it is NaN.
struct RowScale {
  float s, inv;
};
constexpr float kQuantTiny = 7.888609052210118e-31f;  // 2^-100

__device__ __forceinline__ RowScale row_scale(uint32_t max_abs_bits) {
  RowScale r;
  if (max_abs_bits >= 0x7f800000u) {
    r.s = __uint_as_float(0x7fc00000u);
    r.inv = 0.f;
  } else {
    r.s = fmaxf(__uint_as_float(max_abs_bits), kQuantTiny) * (1.0f / 127.0f);
    r.inv = 1.0f / r.s;
  }
  return r;
}

// Eight values to eight signed bytes. v * (1 / s) is off by up to two
// roundings, which can put a value next to a border k + 1/2 on the wrong side;
// the remainder v - q s is exact in fp32 (q has at most 7 bits and the
// remainder is a multiple of an ulp of s or of v not above s/2 by more than a
// few ulp), so it tells: beyond s / 2, or at s / 2 with an odd q, q moves by one.
__device__ __forceinline__ uint2 quant8(const f2 (&v)[4], const RowScale& r) {
  constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23: the sum's low bits are the rounded integer
  const float half = 0.5f * r.s;
  uint32_t t[8];
  float far = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const f2 m = fma2(v[k], both(r.inv), both(kMagic));
    const float2 rem = unpair2(fma2(add2(m, both(-kMagic)), both(-r.s), v[k]));
    far = fmaxf(far, fmaxf(fabsf(rem.x), fabsf(rem.y)));
    const float2 q = unpair2(m);
    t[2 * k] = __float_as_uint(q.x);
    t[2 * k + 1] = __float_as_uint(q.y);
  }
  if (far >= half) {  // rare; false for s = NaN
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float2 p = unpair2(v[e >> 1]);
      const float rem = fmaf(-(__uint_as_float(t[e]) - kMagic), r.s, e & 1 ? p.y : p.x);
      const float ar = fabsf(rem);
      if (ar > half || (ar == half && (t[e] & 1u))) t[e] += rem > 0.f ? 1u : 0xffffffffu;
    }
  }
  if (r.inv == 0.f) {
#pragma unroll
    for (int e = 0; e < 8; ++e) t[e] = 0u;
  }
  uint2 o;
  o.x = __byte_perm(__byte_perm(t[0], t[1], 0x0040), __byte_perm(t[2], t[3], 0x0040), 0x5410);
  o.y = __byte_perm(__byte_perm(t[4], t[5], 0x0040), __byte_perm(t[6], t[7], 0x0040), 0x5410);
  return o;
}

// Largest magnitude of eight values as loaded, as fp32 bits; a NaN stays one, above
// every number.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float max_abs8(const Vec8<float>& r) {
  const float a = max_nan(max_nan(fabsf(r.a.x), fabsf(r.a.y)), max_nan(fabsf(r.a.z), fabsf(r.a.w)));
  const float b = max_nan(max_nan(fabsf(r.b.x), fabsf(r.b.y)), max_nan(fabsf(r.b.z), fabsf(r.b.w)));
  return max_nan(a, b);
}
__device__ __forceinline__ float max_abs8(const Vec8<__nv_bfloat16>& r) {
  const auto h = [](uint32_t w) { return __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w)); };
  const __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(h(r.a.x), h(r.a.y)), __hmax2_nan(h(r.a.z), h(r.a.w)));
  return max_nan(__low2float(m), __high2float(m));
}
__device__ __forceinline__ float max_abs8(const Vec8<__half>& r) {
  const auto h = [](uint32_t w) { return __habs2(*reinterpret_cast<const __half2*>(&w)); };
  const __half2 m = __hmax2_nan(__hmax2_nan(h(r.a.x), h(r.a.y)), __hmax2_nan(h(r.a.z), h(r.a.w)));
  return max_nan(__low2float(m), __high2float(m));
}

}  // namespace mtgr
