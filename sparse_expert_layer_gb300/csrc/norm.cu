// Residual addition, RMS norm and 8-bit codes in one pass over the rows.
//
//   r = x + residual;  y = r * rstd * gamma,  rstd = 1 / sqrt(mean(r^2) + eps)
//   codes of y with one scale per row, or per group of channels.
//
// With v = r * gamma, |y| = rstd * |v|, so a row's (or group's) largest |y| is
// rstd * max|v| and the code of y is the code of v against max|v|: rstd cancels.
// The sum of squares and the largest |v| are therefore one reduction, the row
// stays in registers between it and the stores, and nothing is read twice.
// Sums, v and scales are fp32; the new residual, y and the codes are each
// rounded once, from fp32 values.
//
// Bound by memory for large batches: 8192 x 7168 in bf16 with y and int8 codes
// moves 528 MB in 89 us (5.9 TB/s, 88% of the copy rate), 16384 x 2048 92%; per-
// group scales cost four shuffles a slot (103 us).  Each CTA keeps one row in
// registers and goes on to further rows; what limits the largest rows is the
// instructions between load and store, so conversions are packed, the maximum
// takes two values an instruction and the warp's maximum is one redux.  One row
// of 7168 takes 2.5 us, a launch and two dependent memory round trips.  Rows above
// 16384 channels need 1024 threads of four slots at 64 registers, which spill 88 to
// 344 bytes a thread: 2048 x 32768 with y and int8 codes 140 us in bf16 (64%), 292
// us in fp32 (58%).  Rows that are not whole slots of 16 bytes are read and written
// channel by channel, eight accesses where others take one: 4096 x 7161 bf16 in 93
// us (42%).
#include <math.h>

#include <cuda_fp8.h>

#include <algorithm>

#include "rows.cuh"

namespace moe {

namespace {

constexpr int kNormMaxHidden = 32768;

struct NormArgs {
  const void* x;
  const void* res;    // nullptr: none
  const void* gamma;  // nullptr: ones
  void* sum;          // nullptr: not wanted
  void* y;            // nullptr: not wanted
  void* q;            // nullptr: not wanted
  float* scale;       // [T, groups]
  int64_t ldx, ldr, lds, ldy;
  int T, H, nslots;
  int q_e4m3;         // codes are e4m3 instead of int8
  int q_group;        // channels per scale, 0 = the row
  int groups;
  float eps, inv_h;
};

// The factor from v to its code's value, `most` / amax, as pre * inv: where amax
// is so small that most / amax overflows, v is scaled up by a power of two first.
__device__ __forceinline__ void code_factor(float amax, float most, float* pre, float* inv) {
  *pre = amax < 0x1p-96f ? 0x1p64f : 1.f;
  const float a = amax * *pre;
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(a));
  *inv = a > 0.f ? most * r : 0.f;
}

// Four int8 codes of v * factor, rounded half to even: adding 1.5 * 2^23 leaves
// the rounded integer in the sum's low bits.  |v * factor| is at most 127 +
// rounding, so it needs no clamp; a row with a NaN or an infinity has a NaN (or
// zero) scale, whatever its codes.
__device__ __forceinline__ uint32_t int8_codes(const float* v, float factor) {
  uint32_t u[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) u[j] = __float_as_uint(fmaf(v[j], factor, 12582912.f));
  return __byte_perm(__byte_perm(u[0], u[1], 0x0040), __byte_perm(u[2], u[3], 0x0040), 0x5410);
}
__device__ __forceinline__ uint32_t e4m3_codes(const float* v, float factor) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[0] * factor, v[1] * factor),
                                               __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[2] * factor, v[3] * factor),
                                               __NV_SATFINITE, __NV_E4M3);
  return (lo & 0xffffu) | (hi << 16);
}

// The codes of a slot; factor[j] belongs to its channel j.
template <bool VEC>
__device__ __forceinline__ void store_codes(const NormArgs& a, int t, int s, float (&v)[kSlot],
                                            const float (&pre)[kSlot], const float (&inv)[kSlot]) {
  uint8_t* q = static_cast<uint8_t*>(a.q) + (size_t)t * a.H;
  if constexpr (VEC) {  // one factor: a slot lies inside its group
    if (pre[0] != 1.f) {
#pragma unroll
      for (int j = 0; j < kSlot; ++j) v[j] *= pre[0];
    }
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      w[i] = a.q_e4m3 ? e4m3_codes(v + 4 * i, inv[0]) : int8_codes(v + 4 * i, inv[0]);
    *reinterpret_cast<uint2*>(q + s * kSlot) = make_uint2(w[0], w[1]);
  } else {
    // one after the other: the product of the factors may overflow
#pragma unroll
    for (int j = 0; j < kSlot; ++j) v[j] = v[j] * pre[j] * inv[j];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t w = a.q_e4m3 ? e4m3_codes(v + 4 * i, 1.f) : int8_codes(v + 4 * i, 1.f);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = slot_channel<!VEC>(s, 4 * i + j);
        if (c < a.H) q[c] = (uint8_t)(w >> (8 * j));
      }
    }
  }
}

// Where the threads' sums and maxima of a row meet: per warp, two rows alternate.
struct NormParts {
  float2 part[2][32];
};

// One row from its raw slots on: the new residual, the reduction, y and codes.
// The slots of x (and of the residual) are in rx (rr); `turn` alternates from
// row to row, so that one barrier a row is enough.
template <typename T, int VPT, bool VEC>
__device__ __forceinline__ void norm_row(const NormArgs& a, int t, const Raw8<T> (&rx)[VPT],
                                         const Raw8<T> (&rr)[VPT], NormParts& sh, int& turn) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int nwarps = blockDim.x / 32;
  const float most = a.q_e4m3 ? 448.f : 127.f, unit = a.q_e4m3 ? 1.f / 448.f : 1.f / 127.f;
  float v[VPT][kSlot];
  float ss = 0.f, amax = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int s = threadIdx.x + i * blockDim.x;
#pragma unroll
    for (int j = 0; j < kSlot; ++j) v[i][j] = 0.f;
    if (slot_inside<!VEC>(s, a.nslots)) {
      unpack8<T>(rx[i], v[i]);
      if (a.res) {
        float r[kSlot];
        unpack8<T>(rr[i], r);
#pragma unroll
        for (int j = 0; j < kSlot; ++j) v[i][j] += r[j];
      }
      if (a.sum) store8<T, VEC>(static_cast<T*>(a.sum) + (int64_t)t * a.lds, s, a.H, v[i]);
#pragma unroll
      for (int j = 0; j < kSlot; ++j) ss = fmaf(v[i][j], v[i][j], ss);
      if (a.gamma) {
        float g[kSlot];
        load8<T, VEC>(static_cast<const T*>(a.gamma), s, a.H, g);
#pragma unroll
        for (int j = 0; j < kSlot; ++j) v[i][j] *= g[j];
      }
      amax = max_abs8(amax, v[i]);
    }
  }
  // values >= 0 compare as their bits do; a NaN shows in the sum of squares
  auto all_max = [](float m) {
    return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
  };
  ss = warp_sum(ss);
  amax = all_max(amax);
  if (nwarps > 1) {
    if (lane == 0) sh.part[turn][warp] = make_float2(ss, amax);
    __syncthreads();
    // every warp adds the warps' parts in the same order
    const float2 p = lane < nwarps ? sh.part[turn][lane] : make_float2(0.f, 0.f);
    ss = warp_sum(p.x);
    amax = all_max(p.y);
    turn ^= 1;
  }
  const float mean = fmaf(ss, a.inv_h, a.eps);
  float rstd = rsqrtf(mean);
  // a row of zeros without eps is zeros, not 0 * inf; a finite row whose squares
  // overflowed shows as NaN instead of passing for zeros
  if (mean == 0.f && amax == 0.f) rstd = 0.f;
  if (isinf(mean) && !isinf(amax)) rstd = __int_as_float(0x7fffffff);
  float pre[kSlot], inv[kSlot];
  if (a.q && a.q_group == 0) {
    code_factor(amax, most, &pre[0], &inv[0]);
#pragma unroll
    for (int j = 1; j < kSlot; ++j) {
      pre[j] = pre[0];
      inv[j] = inv[0];
    }
    if (threadIdx.x == 0) a.scale[t] = rstd * amax * unit;
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int s = threadIdx.x + i * blockDim.x;
    const bool inside = slot_inside<!VEC>(s, a.nslots);
    if (a.y && inside) {
      float o[kSlot];
#pragma unroll
      for (int j = 0; j < kSlot; ++j) o[j] = v[i][j] * rstd;
      store8<T, VEC>(static_cast<T*>(a.y) + (int64_t)t * a.ldy, s, a.H, o);
    }
    if (!a.q) continue;
    // a group lies inside a warp's 256 channels (channels past the row are zero)
    if (VEC && a.q_group > 0) {  // the slots of consecutive lanes
      const int lanes = a.q_group / kSlot;
      float m = max_abs8(0.f, v[i]);
      for (int o = lanes / 2; o > 0; o >>= 1)
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      code_factor(m, most, &pre[0], &inv[0]);
      if (inside && lane % lanes == 0)
        a.scale[(size_t)t * a.groups + s / lanes] = rstd * m * unit;
    }
    if (!VEC && a.q_group > 0) {  // channels j of all lanes, for q_group / 32 values of j
      const int each = a.q_group / 32;
      float m[kSlot];
#pragma unroll
      for (int j = 0; j < kSlot; ++j) m[j] = all_max(fabsf(v[i][j]));
#pragma unroll
      for (int o = 1; o < kSlot; o <<= 1)  // over aligned runs of `each`
        if (o < each) {
          float n[kSlot];
#pragma unroll
          for (int j = 0; j < kSlot; ++j) n[j] = fmaxf(m[j], m[j ^ o]);
#pragma unroll
          for (int j = 0; j < kSlot; ++j) m[j] = n[j];
        }
#pragma unroll
      for (int j = 0; j < kSlot; ++j) {
        code_factor(m[j], most, &pre[j], &inv[j]);
        const int c = slot_channel<!VEC>(s, j);
        if (inside && lane == 0 && j % each == 0 && c < a.H)
          a.scale[(size_t)t * a.groups + c / a.q_group] = rstd * m[j] * unit;
      }
    }
    if (inside) store_codes<VEC>(a, t, s, v[i], pre, inv);
  }
}

// blockDim.x threads work on one row, blockDim.y rows at a time; slot s of a
// row belongs to thread s % blockDim.x.
template <typename T, int VPT, bool VEC, int MAXT>
__global__ void __launch_bounds__(MAXT, VPT == 2 && sizeof(T) == 2 ? 2 : 1) add_rmsnorm_kernel(NormArgs a) {
  pdl_enter();
  __shared__ NormParts sh;
  int turn = 0;
  const int step = gridDim.x * blockDim.y;
  for (int t = blockIdx.x * blockDim.y + threadIdx.y; t < a.T; t += step) {
    const T* x = static_cast<const T*>(a.x) + (int64_t)t * a.ldx;
    const T* res = static_cast<const T*>(a.res) + (int64_t)t * a.ldr;
    Raw8<T> rx[VPT], rr[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int s = threadIdx.x + i * blockDim.x;
      if (slot_inside<!VEC>(s, a.nslots)) {
        rx[i] = load_raw8<T, VEC>(x, s, a.H);
        if (a.res) rr[i] = load_raw8<T, VEC>(res, s, a.H);
      }
    }
    norm_row<T, VPT, VEC>(a, t, rx, rr, sh, turn);
    if (t >= a.T - step) break;  // of 2^31 - 1 rows, t + step may lie past an int
  }
}

template <typename T, int VPT, bool VEC, int MAXT>
void launch_as(const Launch& L, const NormArgs& a, int threads, int rows) {
  // a few CTAs' worth of threads on every SM; each goes on to further rows
  const int per_sm = std::max(1, 2048 / (threads * rows));
  const int grid = (int)std::min<int64_t>(((int64_t)a.T + rows - 1) / rows,
                                          (int64_t)L.num_sms * per_sm);
  launch_begin(L, MOE_K_NORM);
  launch_kernel(add_rmsnorm_kernel<T, VPT, VEC, MAXT>, grid, dim3(threads, rows), 0, L.stream, a);
  launch_end(L, MOE_K_NORM);
}

template <typename T, bool VEC>
void launch_norm(const Launch& L, const NormArgs& a) {
  const int slots32 = (a.nslots + 31) / 32;  // warps at one slot a thread
  constexpr bool wide = sizeof(T) == 4;
  if (slots32 <= 32 && (a.T <= L.num_sms || (wide && slots32 <= 16))) {
    // few rows: one slot a thread, the shortest chain from load to store
    // (64 rows of 7168 in bf16: 3.2 us, with two slots 3.6); fp32 rows of up to
    // 4096 fill the SMs that way too (48 against 52 us for 4096 x 4096)
    return launch_as<T, 1, VEC, 1024>(L, a, 32 * slots32, 1);
  }
  if constexpr (!wide) {
    // short rows: a warp holds a row, four rows a CTA
    if (slots32 <= 2) return launch_as<T, 2, VEC, 512>(L, a, 32, 4);
    // two slots: several rows an SM in different phases (8192 x 7168: 89 us)
    if (slots32 <= 32) return launch_as<T, 2, VEC, 512>(L, a, 32 * ((slots32 + 1) / 2), 1);
  }
  if (slots32 <= 64)
    launch_as<T, 4, VEC, 512>(L, a, 32 * ((slots32 + 3) / 4), 1);
  else
    launch_as<T, 4, VEC, 1024>(L, a, 32 * ((slots32 + 3) / 4), 1);
}

template <typename T>
void launch_norm(const Launch& L, const NormArgs& a, bool vec) {
  if (vec)
    launch_norm<T, true>(L, a);
  else
    launch_norm<T, false>(L, a);
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_add_rmsnorm(int32_t T, int32_t H, int32_t dtype, const void* x,
                                      int64_t ldx, const void* residual, int64_t ldr,
                                      const void* gamma, float eps, void* sum, int64_t lds,
                                      void* y, int64_t ldy, int32_t q_dtype, int32_t q_group,
                                      void* q, float* q_scale, moe_stream_t stream) {
  if (T < 0 || H < 1 || !(eps >= 0.f) || !isfinite(eps)) return MOE_ERR_INVALID_ARG;
  if (dtype < MOE_DT_BF16 || dtype > MOE_DT_FP32) return MOE_ERR_INVALID_ARG;
  if (q && q_dtype != MOE_DT_INT8 && q_dtype != MOE_DT_E4M3) return MOE_ERR_INVALID_ARG;
  if (q && q_group != 0 && q_group != 32 && q_group != 64 && q_group != 128 && q_group != 256)
    return MOE_ERR_INVALID_ARG;
  if (H > kNormMaxHidden) return MOE_ERR_UNSUPPORTED;
  if (ldx < H || (residual && ldr < H) || (sum && lds < H) || (y && ldy < H))
    return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!x || (q && !q_scale) || (!sum && !y && !q)) return MOE_ERR_INVALID_ARG;
  if (misaligned16(x, residual, gamma, sum, y, q, q ? q_scale : nullptr)) return MOE_ERR_ALIGNMENT;
  const int es = dtype == MOE_DT_FP32 ? 4 : 2;
  NormArgs a{};
  a.x = x;
  a.res = residual;
  a.gamma = gamma;
  a.sum = sum;
  a.y = y;
  a.q = q;
  a.scale = q_scale;
  a.ldx = ldx;
  a.ldr = ldr;
  a.lds = lds;
  a.ldy = ldy;
  a.T = T;
  a.H = H;
  a.nslots = (H + kSlot - 1) / kSlot;
  a.q_e4m3 = q_dtype == MOE_DT_E4M3;
  a.q_group = q_group;
  a.groups = q_group > 0 ? (H + q_group - 1) / q_group : 1;
  a.eps = eps;
  a.inv_h = 1.f / (float)H;
  // whole slots at 16-byte aligned addresses in every row
  auto whole = [&](const void* p, int64_t ld) { return !p || T == 1 || ld * es % 16 == 0; };
  const bool vec = H % kSlot == 0 && whole(x, ldx) && whole(residual, ldr) && whole(sum, lds) &&
                   whole(y, ldy);
  Launch L;
  moe_status s = open_launch(stream, &L);
  if (s != MOE_OK) return s;
  if (dtype == MOE_DT_BF16)
    launch_norm<__nv_bfloat16>(L, a, vec);
  else if (dtype == MOE_DT_FP16)
    launch_norm<__half>(L, a, vec);
  else
    launch_norm<float>(L, a, vec);
  return launch_status_take();
}
