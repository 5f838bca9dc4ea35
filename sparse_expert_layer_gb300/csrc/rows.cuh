// Row access shared by the operators around the layer (norm.cu, token_sort.cu,
// w4_gemv.cu): a thread owns slots of eight consecutive channels, held in fp32.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"

namespace moe {

constexpr int kSlot = 8;  // channels of one slot

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f<__half>(float v) {
  return __float2half_rn(v);
}

// Eight channels as they lie in memory: one 16-byte word of a 16-bit type, two
// of fp32.
template <typename T>
struct alignas(16) Raw8 {
  uint4 q[sizeof(T) * kSlot / 16];
};

// The slot's raw words.  VEC: the slot is whole and 16-byte aligned.  Otherwise
// its first n (1 .. 8) channels are loaded one by one and the rest are zero.
template <typename T, bool VEC>
__device__ __forceinline__ Raw8<T> load_raw8(const T* p, int n) {
  Raw8<T> r;
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(r.q) / 16); ++i) r.q[i] = reinterpret_cast<const uint4*>(p)[i];
  } else {
    T v[kSlot];
#pragma unroll
    for (int i = 0; i < kSlot; ++i) v[i] = i < n ? p[i] : from_f<T>(0.f);
    memcpy(&r, v, sizeof r);
  }
  return r;
}
template <typename T>
__device__ __forceinline__ void unpack8(const Raw8<T>& r, float (&f)[kSlot]) {
  T v[kSlot];
  memcpy(v, &r, sizeof r);
#pragma unroll
  for (int i = 0; i < kSlot; ++i) f[i] = to_f(v[i]);
}
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* p, int n, float (&f)[kSlot]) {
  unpack8<T>(load_raw8<T, VEC>(p, n), f);
}
// Rounds to nearest even once, here.
template <typename T, bool VEC>
__device__ __forceinline__ void store8(T* p, int n, const float (&f)[kSlot]) {
  T v[kSlot];
#pragma unroll
  for (int i = 0; i < kSlot; ++i) v[i] = from_f<T>(f[i]);
  if constexpr (VEC) {
    Raw8<T> r;
    memcpy(&r, v, sizeof r);
#pragma unroll
    for (int i = 0; i < (int)(sizeof(r.q) / 16); ++i) reinterpret_cast<uint4*>(p)[i] = r.q[i];
  } else {
#pragma unroll
    for (int i = 0; i < kSlot; ++i)
      if (i < n) p[i] = v[i];
  }
}

}  // namespace moe
