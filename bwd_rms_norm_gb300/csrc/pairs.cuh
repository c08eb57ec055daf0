// fp32 arithmetic by pairs (the f32x2 instructions), and the conversion of packed
// 16-bit types to pairs and back.
#pragma once

#include "common.cuh"

namespace rmsn {
namespace {

// Two fp32 values in a 64-bit register.
using f32x2 = unsigned long long;

__device__ __forceinline__ f32x2 pair(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}

__device__ __forceinline__ float2 split(f32x2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}

__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

__device__ __forceinline__ float sum2(f32x2 v) {
  const float2 f = split(v);
  return f.x + f.y;
}

template <typename U>
__device__ __forceinline__ f32x2 widen(uint32_t w);

template <>
__device__ __forceinline__ f32x2 widen<__nv_bfloat16>(uint32_t w) {
  return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

template <>
__device__ __forceinline__ f32x2 widen<__half>(uint32_t w) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  return pair(f.x, f.y);
}

template <typename U>
__device__ __forceinline__ uint32_t narrow(f32x2 v);

template <>
__device__ __forceinline__ uint32_t narrow<__nv_bfloat16>(f32x2 v) {
  const float2 f = split(v);
  const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <>
__device__ __forceinline__ uint32_t narrow<__half>(f32x2 v) {
  const float2 f = split(v);
  const __half2 h = __floats2half2_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// E = 2 N elements of type U at p, 8 or 16 bytes.
template <typename U, int N>
__device__ __forceinline__ void load_pairs(const U* p, f32x2 (&f)[N]) {
  if constexpr (sizeof(U) == 4) {
    static_assert(N == 2, "16 bytes");
    const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(p);
    f[0] = q.x;
    f[1] = q.y;
  } else if constexpr (N == 4) {
    const uint4 q = *reinterpret_cast<const uint4*>(p);
    f[0] = widen<U>(q.x);
    f[1] = widen<U>(q.y);
    f[2] = widen<U>(q.z);
    f[3] = widen<U>(q.w);
  } else {
    static_assert(N == 2, "8 bytes");
    const uint2 q = *reinterpret_cast<const uint2*>(p);
    f[0] = widen<U>(q.x);
    f[1] = widen<U>(q.y);
  }
}

template <typename U, int N>
__device__ __forceinline__ void store_pairs(U* p, const f32x2 (&f)[N]) {
  if constexpr (sizeof(U) == 4) {
    const float2 a = split(f[0]), b = split(f[1]);
    st_vec(p, make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x),
                         __float_as_uint(b.y)));
  } else if constexpr (N == 4) {
    st_vec(p, make_uint4(narrow<U>(f[0]), narrow<U>(f[1]), narrow<U>(f[2]), narrow<U>(f[3])));
  } else {
    *reinterpret_cast<uint2*>(p) = make_uint2(narrow<U>(f[0]), narrow<U>(f[1]));
  }
}

template <int N>
__device__ __forceinline__ float sum_pairs(f32x2 (&f)[N]) {
#pragma unroll
  for (int h = N / 2; h >= 1; h /= 2)
#pragma unroll
    for (int i = 0; i < h; ++i) f[i] = add2(f[i], f[i + h]);
  return sum2(f[0]);
}

}  // namespace
}  // namespace rmsn
