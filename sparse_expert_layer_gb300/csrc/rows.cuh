// Row access shared by the operators around the layer (norm.cu, token_sort.cu,
// w4_gemv.cu): a thread owns slots of eight consecutive channels, held in fp32;
// and copies that run ahead of their use.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"

namespace moe {

constexpr int kSlot = 8;  // channels of one slot

// Slot s of a row of H channels, s = lane modulo 32: channels 8 s .. 8 s + 7, one
// vector access where rows are whole slots at 16-byte boundaries (VEC).  SPREAD,
// for other rows: the 32 slots of a warp share 256 channels and a slot takes every
// 32nd of them, so that a warp's element-wise accesses lie side by side (4096 rows
// of 7161 through the norm: 191 us with eight neighbours a thread).
template <bool SPREAD>
__device__ __forceinline__ int slot_channel(int s, int j) {
  return SPREAD ? (s & ~31) * kSlot + j * 32 + (s & 31) : s * kSlot + j;
}
// Whether slot s has any channel of the row's nslots slots.
template <bool SPREAD>
__device__ __forceinline__ bool slot_inside(int s, int nslots) {
  return (SPREAD ? s & ~31 : s) < nslots;
}

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

// The raw words of slot s of a row (channels past H are zero).
template <typename T, bool VEC, bool SPREAD = !VEC>
__device__ __forceinline__ Raw8<T> load_raw8(const T* row, int s, int H) {
  Raw8<T> r;
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(r.q) / 16); ++i)
      r.q[i] = reinterpret_cast<const uint4*>(row + s * kSlot)[i];
  } else {
    T v[kSlot];
#pragma unroll
    for (int j = 0; j < kSlot; ++j) {
      const int c = slot_channel<SPREAD>(s, j);
      v[j] = c < H ? row[c] : from_f<T>(0.f);
    }
    memcpy(&r, v, sizeof r);
  }
  return r;
}
// Two 16-bit values of one word to fp32 and back (rounded to nearest even).
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
  return make_float2(bf16lo(w), bf16hi(w));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
  __half2 h;
  memcpy(&h, &w, 4);
  return __half22float2(h);
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  uint32_t w;
  memcpy(&w, &h, 4);
  return w;
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  uint32_t w;
  memcpy(&w, &h, 4);
  return w;
}

template <typename T>
__device__ __forceinline__ void unpack8(const Raw8<T>& r, float (&f)[kSlot]) {
  if constexpr (sizeof(T) == 4) {
    memcpy(f, &r, sizeof r);
  } else {
    const uint32_t w[4] = {r.q[0].x, r.q[0].y, r.q[0].z, r.q[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = unpack2<T>(w[i]);
      f[2 * i] = v.x;
      f[2 * i + 1] = v.y;
    }
  }
}
template <typename T>
__device__ __forceinline__ Raw8<T> pack8(const float (&f)[kSlot]) {
  Raw8<T> r;
  if constexpr (sizeof(T) == 4)
    memcpy(&r, f, sizeof r);
  else
    r.q[0] = make_uint4(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]), pack2<T>(f[4], f[5]),
                        pack2<T>(f[6], f[7]));
  return r;
}
template <typename T, bool VEC, bool SPREAD = !VEC>
__device__ __forceinline__ void load8(const T* row, int s, int H, float (&f)[kSlot]) {
  unpack8<T>(load_raw8<T, VEC, SPREAD>(row, s, H), f);
}
// Rounds to nearest even once, here.
template <typename T, bool VEC, bool SPREAD = !VEC>
__device__ __forceinline__ void store8(T* row, int s, int H, const float (&f)[kSlot]) {
  const Raw8<T> r = pack8<T>(f);
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(r.q) / 16); ++i)
      reinterpret_cast<uint4*>(row + s * kSlot)[i] = r.q[i];
  } else {
    T v[kSlot];
    memcpy(v, &r, sizeof r);
#pragma unroll
    for (int j = 0; j < kSlot; ++j) {
      const int c = slot_channel<SPREAD>(s, j);
      if (c < H) row[c] = v[j];
    }
  }
}

// max(m, |f[0]|, ..., |f[7]|), two values an instruction.
__device__ __forceinline__ float max_abs8(float m, const float (&f)[kSlot]) {
#pragma unroll
  for (int i = 0; i < kSlot; i += 2)
    asm("max.abs.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(f[i]), "f"(f[i + 1]));
  return m;
}

// ------------------------------------------------ asynchronous row copies ----
// Global -> shared by the calling thread, past the L1; waited for by groups.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// real false: the 16 bytes become zeros, src is not read
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(real ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_unit(uint32_t dst, const void* src, int bytes) {
  if (bytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else if (bytes == 8)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
}  // namespace moe
