// The expert layer for at most eight tokens, in two kernels: router and top-k, then
// every picked expert's SwiGLU FFN with the weighted combine.
//
//   out[t] = sum over picks j of w[t, j] * (expert e: W_d (silu(W_g x_t) * (W_u x_t));
//            zero-computation expert: x_t) + shared expert(x_t)
//
// Bound by the weights of the distinct picked experts, each read once: with a few
// tokens hardly any expert has more than one, so all products are 16-row MMA tiles of
// weights (m16n8k16) against up to eight columns, and the columns are the tokens
// themselves.  A column of a token that did not pick the expert is computed all the
// same and dropped (gate and up) or zero (down); nothing is sorted or gathered, and a
// token that is not finite stays in its column.
//
// The second kernel has one CTA an SM.  Gate and up: teams of four warps claim tiles of
// 8 or 16 channels of an expert (8 gate and 8 up rows an MMA tile), a quarter of K a
// warp; their parts are added in order, SwiGLU gives h in fp32.  Down: a CTA owns a
// range of output channels of all experts; its 16 warps split the (expert, K) steps
// evenly, apply the routing weights to their own sums, and add them in order: one
// rounded store, no atomics, the same bits on every call.  Between the two a CTA waits
// until all tiles have stored h.  Tiles are claimed, so a tile that a waiting CTA needs
// belongs to a running team, whatever else occupies the GPU; and the first stages of
// the down weights are on their way during the wait.  Every warp streams its weights
// through a cp.async ring of its own, so nothing but a tile's sum needs a barrier.
//
// 4-bit weights: a nibble alone in the low bits of a half is the fp16 subnormal
// q * 2^-24 (four bits up: q * 2^-20, its x is divided by 16), so a weight costs part of
// one AND.  x (and h) are scaled by a power of two for each token that brings their
// largest value to 2^13, which makes them fp16 exactly (bf16 values: down to 2^-26 of
// the largest), h rounded to 11 bits.  A block's sum of (q - z) x is 2^24 times the
// MMA's sum minus z times the sum of x, which a further MMA of ones gives for h; scales
// are applied in fp32.  16-bit weights: x as it is, h as a sum of two 16-bit numbers.
#include <math.h>

#include "few_plan.h"
#include "mma.cuh"
#include "topk.cuh"

namespace moe {

namespace {

constexpr int kFewThreads = 32 * kFewWarps;
constexpr int kRouteThreads = 256;
constexpr int kRouteWarps = kRouteThreads / 32;
constexpr int kFewMaxPicks = kFewMaxT * 32;
constexpr int kFewMaxTH = 65536;           // tokens x hidden
constexpr int kRouteScratch = 96 * 1024;   // top-k scratch in shared memory, at most
constexpr int kRouteSmem = 212 * 1024;     // eight rows for five tokens of kFewMaxTH / 5

// One expert with rows (expert -1: the shared one).
struct FewUnit {
  int expert;
  uint32_t tokens;    // bit t: token t picked it
  float w[kFewMaxT];  // its routing weight, 0 for other tokens
};
static_assert(sizeof(FewUnit) == kFewUnitBytes, "the plan's size");

// Workspace after the status block.  `ticket` is zero between calls; the rest is
// written by the first kernel.
struct FewHead {
  int ticket;
  int claim, done;  // gate/up tiles claimed and stored
  int units;        // without the shared one
  float zero_w[kFewMaxT];  // weights of the tokens' zero-computation picks
  FewUnit unit[kFewMaxPicks + 1];
  uint32_t hmax[kFewMaxPicks + 1][kFewMaxT];  // largest |h| of a unit's token, fp32 bits
};

struct FewMatrix {
  const unsigned char* w;
  const unsigned char* s;
  const unsigned char* z;
};

struct FewArgs {
  const void* x;
  int64_t ldx;
  void* out;
  int64_t ldo;
  FewMatrix m[3], shared[3];  // gate, up, down
  FewHead* head;
  DevStatus* status;
  float* h;  // [unit][token][inter]
  int T, H, I, Is, inter;
  int fp16, vec;  // type of x and out; rows of x in 16-byte pieces
  int group, scale_dtype;
  FewPlan p;
};

struct RouteArgs {
  TopkArgs tk;
  const void* x;
  int64_t ldx;
  const float* w_r;
  float* logits;   // [T, E]
  float* scratch;  // 3 E floats a token, where shared memory has no room
  int32_t* ids;    // outputs, or nullptr
  float* w;
  FewHead* head;
  int H, E_r, shared, fp16, vec;
};

// ---------------------------------------------------------------- routing ----
__device__ __forceinline__ float2 unpack_x(uint32_t w, int fp16) {
  return fp16 ? unpack2<__half>(w) : unpack2<__nv_bfloat16>(w);
}
// Eight channels of a 16-bit row.
__device__ __forceinline__ uint4 load_x8(const void* x, int64_t at, bool vec) {
  const uint16_t* p = static_cast<const uint16_t*>(x) + at;
  if (vec) return *reinterpret_cast<const uint4*>(p);
  uint16_t v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = p[i];
  uint4 q;
  memcpy(&q, v, 16);
  return q;
}

// Logits of the CTA's experts for all TT >= T tokens; the last CTA picks.
template <int TT>
__global__ void __launch_bounds__(kRouteThreads) few_route_kernel(RouteArgs a) {
  pdl_enter();
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ float part[kRouteWarps][2][TT];
  __shared__ int32_t ids[kFewMaxPicks];
  __shared__ float wts[kFewMaxPicks];
  __shared__ int warp_units[kRouteWarps];
  __shared__ int last;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int T = a.tk.T, H = a.H, E = a.tk.E, k = a.tk.k;
  for (int i = tid; i < TT * (H / 8); i += kRouteThreads) {
    const int t = i / (H / 8), c = i % (H / 8);
    reinterpret_cast<uint4*>(smem)[i] =
        t < T ? load_x8(a.x, t * a.ldx + 8 * c, a.vec) : make_uint4(0u, 0u, 0u, 0u);
  }
  __syncthreads();
  constexpr int kCols = 4;  // float4 of each row in flight
  for (int r = blockIdx.x; r < E; r += 2 * gridDim.x) {
    const bool two = r + gridDim.x < E;
    const float4* w0 = reinterpret_cast<const float4*>(a.w_r + (size_t)r * H);
    const float4* w1 = reinterpret_cast<const float4*>(
        a.w_r + (size_t)(two ? r + gridDim.x : r) * H);
    float acc[2][TT] = {};
    for (int c0 = tid; c0 < H / 4; c0 += kCols * kRouteThreads) {
      float4 v0[kCols], v1[kCols];
#pragma unroll
      for (int i = 0; i < kCols; ++i) {
        const int c = c0 + i * kRouteThreads;
        v0[i] = c < H / 4 ? __ldg(w0 + c) : make_float4(0.f, 0.f, 0.f, 0.f);
        v1[i] = c < H / 4 && two ? __ldg(w1 + c) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int i = 0; i < kCols; ++i) {
        const int c = c0 + i * kRouteThreads;
        if (c >= H / 4) break;
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          const uint2 q = reinterpret_cast<const uint2*>(smem)[t * (H / 4) + c];
          const float2 x0 = unpack_x(q.x, a.fp16), x1 = unpack_x(q.y, a.fp16);
          acc[0][t] = fmaf(v0[i].x, x0.x, acc[0][t]);
          acc[0][t] = fmaf(v0[i].y, x0.y, acc[0][t]);
          acc[0][t] = fmaf(v0[i].z, x1.x, acc[0][t]);
          acc[0][t] = fmaf(v0[i].w, x1.y, acc[0][t]);
          acc[1][t] = fmaf(v1[i].x, x0.x, acc[1][t]);
          acc[1][t] = fmaf(v1[i].y, x0.y, acc[1][t]);
          acc[1][t] = fmaf(v1[i].z, x1.x, acc[1][t]);
          acc[1][t] = fmaf(v1[i].w, x1.y, acc[1][t]);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        const float v = warp_sum(acc[j][t]);
        if (lane == 0) part[warp][j][t] = v;
      }
    __syncthreads();
    if (tid < 2 * TT) {
      const int j = tid / TT, t = tid % TT;
      float v = 0.f;
#pragma unroll
      for (int i = 0; i < kRouteWarps; ++i) v += part[i][j][t];
      if (t < T && (j == 0 || two)) a.logits[(size_t)t * E + r + j * gridDim.x] = v;
    }
    __syncthreads();
  }
  if (tid == 0) {
    __threadfence();
    last = atomicAdd(&a.head->ticket, 1) == (int)gridDim.x - 1;
    __threadfence();
  }
  __syncthreads();
  if (!last) return;

  // Picks of all tokens, a warp each.
  float* lg = reinterpret_cast<float*>(smem);
  const bool inside = T * E * 16 <= kRouteScratch;
  for (int i = tid; i < T * E && inside; i += kRouteThreads) lg[i] = __ldcg(a.logits + i);
  for (int i = tid; i < T * k; i += kRouteThreads) ids[i] = -1;
  __syncthreads();
  if (warp < T) {
    TopkArgs tk = a.tk;
    tk.ids = ids;
    tk.w = wts;
    const float* row = inside ? lg + warp * E : a.logits + (size_t)warp * E;
    float* scratch = inside ? lg + T * E + warp * 3 * E : a.scratch + (size_t)warp * 3 * E;
    topk_token(tk, warp, row, scratch);
  }
  __syncthreads();

  // Units: the distinct experts with weights, in order of their first pick.
  FewHead* head = a.head;
  const int picks = T * k;
  const int e = tid < picks ? ids[tid] : -1;
  bool first = e >= 0 && e < a.E_r;
  for (int i = 0; i < tid && first; ++i) first = ids[i] != e;
  const uint32_t ballot = __ballot_sync(0xffffffffu, first);
  if (lane == 0) warp_units[warp] = __popc(ballot);
  __syncthreads();
  int before = 0, units = 0;
  for (int i = 0; i < kRouteWarps; ++i) {
    before += i < warp ? warp_units[i] : 0;
    units += warp_units[i];
  }
  if (first) {
    FewUnit u;
    u.expert = e;
    u.tokens = 0u;
#pragma unroll
    for (int t = 0; t < kFewMaxT; ++t) u.w[t] = 0.f;
    for (int i = tid; i < picks; ++i)
      if (ids[i] == e) {
        u.tokens |= 1u << (i / k);
#pragma unroll
        for (int t = 0; t < kFewMaxT; ++t)
          if (t == i / k) u.w[t] += wts[i];
      }
    head->unit[before + __popc(ballot & ((1u << lane) - 1u))] = u;
  }
  if (tid < kFewMaxT) {
    float z = 0.f;
    for (int j = 0; j < k && tid < T; ++j)
      if (ids[tid * k + j] >= a.E_r) z += wts[tid * k + j];
    head->zero_w[tid] = z;
  }
  if (tid == 0) {
    if (a.shared) {
      FewUnit u;
      u.expert = -1;
      u.tokens = (1u << T) - 1u;
#pragma unroll
      for (int t = 0; t < kFewMaxT; ++t) u.w[t] = t < T ? 1.f : 0.f;
      head->unit[units] = u;
    }
    head->units = units;
    head->ticket = head->claim = head->done = 0;
  }
  for (int i = tid; i < (units + 1) * kFewMaxT; i += kRouteThreads)
    (&head->hmax[0][0])[i] = 0u;
  for (int i = tid; i < picks; i += kRouteThreads) {
    if (a.ids) a.ids[i] = ids[i];
    if (a.w) a.w[i] = wts[i];
  }
}

// ------------------------------------------------------------------- FFN ----
__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(at)
               : "memory");
  return v;
}
// The first n (0 .. 4) bytes of a word, zeros after them.
__device__ __forceinline__ void cp_async_word(uint32_t dst, const void* src, int n) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void team_barrier(int team) {
  asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "n"(32 * kFewTeamWarps) : "memory");
}
// All but the `stages - 2` groups committed last have arrived.
__device__ __forceinline__ void wait_stage(int stages) {
  switch (stages) {
    case 2: cp_async_wait<0>(); break;
    case 3: cp_async_wait<1>(); break;
    case 4: cp_async_wait<2>(); break;
    case 5: cp_async_wait<3>(); break;
    case 6: cp_async_wait<4>(); break;
    case 7: cp_async_wait<5>(); break;
    default: cp_async_wait<6>(); break;
  }
}

__device__ __forceinline__ float read_scale(uint32_t at, int dtype) {
  if (dtype == MOE_DT_FP32) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
  }
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at) : "memory");
  return dtype == MOE_DT_BF16 ? bf16_to_f(v) : __half2float(__ushort_as_half(v));
}
__device__ __forceinline__ float read_zero(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return (float)(v & 31u);
}

// Where a lane's two weight rows of a 16-row tile have their groups: the byte of a
// stage's first group inside its first word (bits 0-1 of the row's address).
struct FewSkew {
  uint32_t s, z;  // address of the first row's first group, modulo 4
  uint32_t s8, z8;
};

// The kinds of weights.  kWords: granules of eight K that a lane supplies in a stage;
// granule i is x's 16-byte piece granule(i, tg) of the stage.
template <int BLOCK, bool ZEROS>
struct Four {
  using Mma = __half;
  static constexpr bool kFour = true, kZeros = ZEROS, kScaled = true, kRest = false;
  static constexpr int kStepK = 256, kWords = 8;
  static constexpr int kBlock = BLOCK, kBlocks = 256 / BLOCK, kPer = BLOCK / 32;
  // first K of granule i of quad lane tg
  static __device__ __forceinline__ int k_of(int i, int tg) {
    return (i / kPer) * BLOCK + tg * (BLOCK / 4) + (i % kPer) * 8;
  }
  // its piece of x: the four lanes of a quad side by side
  static __device__ __forceinline__ int piece(int i, int tg) {
    return (i / kPer) * (BLOCK / 8) + (i % kPer) * 4 + tg;
  }
  static __device__ __forceinline__ int piece_of_k8(int j) {  // granule j = K / 8
    const int b = j / (BLOCK / 8), r = j % (BLOCK / 8);
    return b * (BLOCK / 8) + (r % kPer) * 4 + r / kPer;
  }
  // 16-byte chunk c of row r lies at chunk swizzle(r, c): the rows that a load meets
  // at once lie side by side in the banks
  static __device__ __forceinline__ int swizzle(int r, int c) {
    return BLOCK == 128 ? c ^ ((r & 1) << 2) : BLOCK == 64 ? c ^ ((r & 3) << 1) : c ^ (r & 7);
  }
  // (k0, k4) (k1, k5) / 16 (k2, k6) (k3, k7) / 16 of eight values
  static __device__ __forceinline__ void operands(const float (&v)[8], uint32_t (&b)[4]) {
    b[0] = pack2<__half>(v[0], v[4]);
    b[1] = pack2<__half>(v[1] * 0.0625f, v[5] * 0.0625f);
    b[2] = pack2<__half>(v[2], v[6]);
    b[3] = pack2<__half>(v[3] * 0.0625f, v[7] * 0.0625f);
  }
};
template <typename T>
struct Sixteen {
  using Mma = T;
  static constexpr bool kFour = false, kRest = true;
  static constexpr bool kScaled = std::is_same<T, __half>::value;  // h needs fp16's range
  static constexpr int kStepK = 64, kWords = 2;
  static constexpr int kBlocks = 1;
  static __device__ __forceinline__ int k_of(int i, int tg) { return i * 32 + tg * 8; }
  static __device__ __forceinline__ int piece(int i, int tg) { return i * 4 + tg; }
  static __device__ __forceinline__ int piece_of_k8(int j) { return j; }
  static __device__ __forceinline__ int swizzle(int r, int c) { return c ^ ((r & 1) << 2); }
};

// acc += a stage's 16 rows times b.  xs: sums of x over the stage's blocks for the
// lane's columns 2 tg and 2 tg + 1.
template <typename K>
__device__ __forceinline__ void multiply(uint32_t st, const uint32_t (&b)[K::kWords][4],
                                         const uint32_t (&rest)[K::kRest ? K::kWords : 1][4],
                                         const float2 (&xs)[K::kBlocks], bool with_rest,
                                         const FewArgs& a, const FewSkew& skew, int step,
                                         float (&acc)[4]) {
  const int lane = threadIdx.x % 32, g = lane / 4, tg = lane % 4;
  const uint32_t row = st + g * 128;
  if constexpr (K::kFour) {
    const uint32_t sbase = st + kFewSub, zbase = sbase + 64 * a.p.swords;
    const int es = a.scale_dtype == MOE_DT_FP32 ? 4 : 2;
    // groups of a stage; 0: one for the whole row
    const int gs = a.group ? K::kBlocks : 0;
    const uint32_t s0 = sbase + g * 4 * a.p.swords + ((skew.s + step * gs * es) & 3u);
    const uint32_t s8 = sbase + (g + 8) * 4 * a.p.swords + ((skew.s8 + step * gs * es) & 3u);
    const uint32_t z0 = zbase + g * 4 * a.p.zwords + ((skew.z + step * gs) & 3u);
    const uint32_t z8 = zbase + (g + 8) * 4 * a.p.zwords + ((skew.z8 + step * gs) & 3u);
#pragma unroll
    for (int blk = 0; blk < K::kBlocks; ++blk) {
      uint32_t lo[K::kPer], hi[K::kPer];
      const int byte = blk * (K::kBlock / 2) + tg * (K::kBlock / 8);
      const uint32_t at = row + K::swizzle(g, byte / 16) * 16 + byte % 16;
      if constexpr (K::kPer == 4) {
        const uint4 u = lds128(at), v = lds128(at + 8 * 128);
        lo[0] = u.x, lo[1] = u.y, lo[2] = u.z, lo[3] = u.w;
        hi[0] = v.x, hi[1] = v.y, hi[2] = v.z, hi[3] = v.w;
      } else if constexpr (K::kPer == 2) {
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(lo[0]), "=r"(lo[1]) : "r"(at) : "memory");
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                     : "=r"(hi[0]), "=r"(hi[1]) : "r"(at + 8 * 128) : "memory");
      } else {
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(lo[0]) : "r"(at) : "memory");
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(hi[0]) : "r"(at + 8 * 128) : "memory");
      }
      float d[4] = {};
#pragma unroll
      for (int i = 0; i < K::kPer; ++i) {
        const int w = blk * K::kPer + i;
        const uint32_t l = lo[i], h = hi[i], l8 = l >> 8, h8 = h >> 8;
        mma16816<__half>(d, l & 0x000f000fu, h & 0x000f000fu, l & 0x00f000f0u, h & 0x00f000f0u,
                         b[w][0], b[w][1]);
        mma16816<__half>(d, l8 & 0x000f000fu, h8 & 0x000f000fu, l8 & 0x00f000f0u,
                         h8 & 0x00f000f0u, b[w][2], b[w][3]);
      }
      const int j = gs ? blk : 0;
      const float sa = read_scale(s0 + j * es, a.scale_dtype);
      const float sb = read_scale(s8 + j * es, a.scale_dtype);
      const float za = K::kZeros ? read_zero(z0 + j) : 8.f;
      const float zb = K::kZeros ? read_zero(z8 + j) : 8.f;
      constexpr float kUp = 16777216.f;
      acc[0] = fmaf(sa, fmaf(d[0], kUp, -za * xs[blk].x), acc[0]);
      acc[1] = fmaf(sa, fmaf(d[1], kUp, -za * xs[blk].y), acc[1]);
      acc[2] = fmaf(sb, fmaf(d[2], kUp, -zb * xs[blk].x), acc[2]);
      acc[3] = fmaf(sb, fmaf(d[3], kUp, -zb * xs[blk].y), acc[3]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < K::kWords; ++i) {
      const uint32_t at = row + K::swizzle(g, i * 4 + tg) * 16;
      const uint4 u = lds128(at), v = lds128(at + 8 * 128);
      mma16816<typename K::Mma>(acc, u.x, v.x, u.y, v.y, b[i][0], b[i][1]);
      mma16816<typename K::Mma>(acc, u.z, v.z, u.w, v.w, b[i][2], b[i][3]);
      if (with_rest) {
        mma16816<typename K::Mma>(acc, u.x, v.x, u.y, v.y, rest[i][0], rest[i][1]);
        mma16816<typename K::Mma>(acc, u.z, v.z, u.w, v.w, rest[i][2], rest[i][3]);
      }
    }
  }
}

// Sizes of one of the layer's matrices: rows of `row` bytes, `groups` scales each.
struct FewShape {
  int K, steps, row, groups;
};
template <typename K>
__device__ __forceinline__ FewShape shape_of(const FewArgs& a, int k) {
  FewShape s;
  s.K = k;
  s.steps = (k + K::kStepK - 1) / K::kStepK;
  s.row = K::kFour ? k / 2 : k * 2;
  s.groups = a.group ? k / a.group : 1;
  return s;
}

// Copies a stage: 16 rows of 128 bytes (zeros past the row's end), and their scales and
// zero points.  wp[i]: the lane's row lane / 8 + 4 i of the tile; sp, zp: the scales of row
// lane / 2, up to send, zend.
template <typename K>
__device__ __forceinline__ void copy_stage(const FewArgs& a, const FewShape& sh, uint32_t st,
                                           int step, const unsigned char* const (&wp)[4],
                                           const unsigned char* sp, const unsigned char* zp) {
  const int lane = threadIdx.x % 32;
  const int byte = step * 128 + (lane % 8) * 16;
  const bool in = byte < sh.row;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = lane / 8 + 4 * i;
    cp_async16_or_zero(st + r * 128 + K::swizzle(r, lane % 8) * 16, wp[i] + (in ? byte : 0), in);
  }
  if constexpr (K::kFour) {
    const int es = a.scale_dtype == MOE_DT_FP32 ? 4 : 2;
    const int gs = a.group ? K::kBlocks : 0;
    auto words = [&](const unsigned char* row, int first, int end, int n, uint32_t dst) {
      const uintptr_t at = reinterpret_cast<uintptr_t>(row + first) & ~(uintptr_t)3;
      const uintptr_t stop = reinterpret_cast<uintptr_t>(row + end);
      for (int i = lane % 2; i < n; i += 2) {
        const uintptr_t p = at + 4 * i;
        const int left = p < stop ? (int)min((uintptr_t)4, stop - p) : 0;
        cp_async_word(dst + (lane / 2) * 4 * n + 4 * i,
                      reinterpret_cast<const void*>(left ? p : (at & ~(uintptr_t)3)), left);
      }
    };
    words(sp, min(step * gs, sh.groups - 1) * es, sh.groups * es, a.p.swords, st + kFewSub);
    if constexpr (K::kZeros)
      words(zp, min(step * gs, sh.groups - 1), sh.groups, a.p.zwords,
            st + kFewSub + 64 * a.p.swords);
  }
}

// Parts of the gate/up tiles' numbering.
struct FewTiles {
  int routed, shared;  // tiles of one routed expert, of the shared one
  int units, total;
};
__device__ __forceinline__ void tile_at(const FewTiles& n, int tile, int* unit, int* first) {
  if (tile < n.units * n.routed) {
    *unit = tile / n.routed;
    *first = tile % n.routed;
  } else {
    *unit = n.units;
    *first = tile - n.units * n.routed;
  }
}

template <typename K, int MT>
__device__ __forceinline__ void gate_up(const FewArgs& a, unsigned char* smem, const FewUnit* units,
                                        const FewTiles& n, const float* x_inverse) {
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int team = warp / kFewTeamWarps, kw = warp % kFewTeamWarps, tt = tid % (32 * kFewTeamWarps);
  const int g = lane / 4, tg = lane % 4;
  const FewShape sh = shape_of<K>(a, a.H);
  const int per = (sh.steps + kFewTeamWarps - 1) / kFewTeamWarps;
  const int k0 = min(sh.steps, kw * per), k1 = min(sh.steps, k0 + per);
  const int S = a.p.stages;
  // tiles a team knows beyond the one it works on: as many as its rings reach into
  const int least = sh.steps - (sh.steps - 1) / per * per;  // the last busy warp's steps
  const int ahead = (S - 1 + least * MT - 1) / (least * MT);
  volatile int* queue = reinterpret_cast<int*>(smem + a.p.queue_at) + team * 16;
  float* red = reinterpret_cast<float*>(smem + a.p.red_at) + team * kFewTeamWarps * MT * 128;
  const uint32_t ring = smem_u32(smem) + a.p.ring_at + warp * S * a.p.sub_bytes;
  FewHead* head = a.head;
  if (tt == 0) {
    const int base = atomicAdd(&head->claim, ahead + 1);
    for (int i = 0; i <= ahead; ++i) queue[i] = base + i;
  }
  team_barrier(team);

  // what is copied next: stage (step, m) of tile queue[seq]
  struct {
    int seq, step, m;
    bool fresh, done;
    const unsigned char* gate;  // the lane's row lane / 8 of the tile's first gate rows
    const unsigned char* up;
    const unsigned char* s;     // scales and zero points of the lane's row lane / 2
    const unsigned char* z;
    int last;  // the most eight-row blocks the tile may go on
  } next{0, k0, 0, true, k0 == k1, nullptr, nullptr, nullptr, nullptr, 0};
  uint32_t fill = 0;
  auto issue = [&]() {
    if (!next.done && next.fresh) {
      const int tile = queue[next.seq % 16];
      next.done = tile >= n.total;
      if (!next.done) {
        int u, f;
        tile_at(n, tile, &u, &f);
        const int e = units[u].expert, N = e < 0 ? a.Is : a.I;
        const FewMatrix* m = e < 0 ? a.shared : a.m;
        const int64_t row = (e < 0 ? 0 : (int64_t)e * N) + f * 8 * MT;
        next.last = (N - f * 8 * MT) / 8 - 1;
        next.gate = m[0].w + (row + lane / 8) * sh.row;
        next.up = m[1].w + (row + lane / 8) * sh.row;
        if constexpr (K::kFour) {
          const FewMatrix& mine = m[lane / 16];  // rows 0-7 of a tile are gate's
          const int es = a.scale_dtype == MOE_DT_FP32 ? 4 : 2;
          next.s = mine.s + (row + lane / 2 % 8) * sh.groups * es;
          if constexpr (K::kZeros) next.z = mine.z + (row + lane / 2 % 8) * sh.groups;
        }
        next.fresh = false;
      }
    }
    if (!next.done) {
      const int64_t skip = min(next.m, next.last) * 8;
      const unsigned char* const wp[4] = {
          next.gate + skip * sh.row, next.gate + (skip + 4) * sh.row, next.up + skip * sh.row,
          next.up + (skip + 4) * sh.row};
      const int es = a.scale_dtype == MOE_DT_FP32 ? 4 : 2;
      copy_stage<K>(a, sh, ring + fill, next.step, wp, next.s + skip * sh.groups * es,
                    next.z + skip * sh.groups);
      if (++next.m == MT) {
        next.m = 0;
        if (++next.step == k1) {
          next.step = k0;
          ++next.seq;
          next.fresh = true;
        }
      }
    }
    cp_async_commit();
    fill = fill == (uint32_t)(S - 1) * a.p.sub_bytes ? 0u : fill + a.p.sub_bytes;
  };
  for (int i = 0; i < S - 1; ++i) issue();

  uint32_t use = 0;
  const uint32_t xrow = smem_u32(smem) + min(g, a.T - 1) * a.p.xpitch;
  const uint32_t sums = smem_u32(smem) + a.p.sum_at + tg * 8;
  for (int seq = 0;; ++seq) {
    const int tile = queue[seq % 16];
    if (tile >= n.total) break;
    int claimed = 0;
    if (tt == 0) claimed = atomicAdd(&head->claim, 1);
    int u, f;
    tile_at(n, tile, &u, &f);
    const int e = units[u].expert, N = e < 0 ? a.Is : a.I;
    const int64_t row0 = (e < 0 ? 0 : (int64_t)e * N) + f * 8 * MT + g;
    const uint32_t es = a.scale_dtype == MOE_DT_FP32 ? 4 : 2;
    float acc[MT][4] = {};
    for (int step = k0; step < k1; ++step) {
      uint32_t b[K::kWords][4];
      float2 xs[K::kBlocks];
#pragma unroll
      for (int i = 0; i < K::kWords; ++i) {
        const uint4 v = lds128(xrow + (step * (K::kStepK / 8) + K::piece(i, tg)) * 16);
        b[i][0] = v.x, b[i][1] = v.y, b[i][2] = v.z, b[i][3] = v.w;
      }
      if constexpr (K::kFour) {
#pragma unroll
        for (int i = 0; i < K::kBlocks; ++i)
          asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];"
                       : "=f"(xs[i].x), "=f"(xs[i].y)
                       : "r"(sums + (step * K::kBlocks + i) * kFewMaxT * 4)
                       : "memory");
      }
      const uint32_t none[K::kRest ? K::kWords : 1][4] = {};
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        wait_stage(S);
        __syncwarp();
        issue();
        const int64_t row = row0 + min(m, (N - f * 8 * MT) / 8 - 1) * 8;
        FewSkew skew{};
        if constexpr (K::kFour) {
          skew.s = skew.s8 = (uint32_t)(row * sh.groups * es);
          skew.z = skew.z8 = (uint32_t)(row * sh.groups);
        }
        multiply<K>(ring + use, b, none, xs, false, a, skew, step, acc[m]);
        use = use == (uint32_t)(S - 1) * a.p.sub_bytes ? 0u : use + a.p.sub_bytes;
      }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      float* r = red + (kw * MT + m) * 128 + g * 8 + 2 * tg;
      *reinterpret_cast<float2*>(r) = make_float2(acc[m][0], acc[m][1]);
      *reinterpret_cast<float2*>(r + 64) = make_float2(acc[m][2], acc[m][3]);
    }
    if (tt == 0) queue[(seq + ahead + 1) % 16] = claimed;
    team_barrier(team);
    if (tt < 64 * MT) {
      const int ch = tt % 8, t = tt / 8 % 8, m = tt / 64;
      const int c = f * 8 * MT + m * 8 + ch;
      float gate = 0.f, up = 0.f;
#pragma unroll
      for (int i = 0; i < kFewTeamWarps; ++i) {
        gate += red[(i * MT + m) * 128 + ch * 8 + t];
        up += red[(i * MT + m) * 128 + (ch + 8) * 8 + t];
      }
      const bool mine = c < N && ((units[u].tokens >> t) & 1u);
      float h = 0.f;
      if (mine) {
        if constexpr (K::kFour) {
          gate *= x_inverse[t];
          up *= x_inverse[t];
        }
        h = gate / (1.f + expf(-gate)) * up;
        __stcg(a.h + ((int64_t)u * a.T + t) * a.inter + c, h);
      }
      if constexpr (K::kScaled) {
        uint32_t most = __float_as_uint(fabsf(h));
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
        if (ch == 0 && mine) atomicMax(&head->hmax[u][t], most);
      }
    }
    team_barrier(team);
    if (tt == 0) {
      __threadfence();
      atomicAdd(&head->done, 1);
    }
  }
  cp_async_wait<0>();
}

constexpr int kFewDownTiles = 4;  // 16-row tiles of one pass of the down projection

template <typename K>
__device__ __forceinline__ void down(const FewArgs& a, unsigned char* smem, const FewUnit* units,
                                     const FewTiles& n, bool shared, const float* zero_w) {
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int g = lane / 4, tg = lane % 4;
  const FewShape rs = shape_of<K>(a, a.I), ss = shape_of<K>(a, a.Is);
  const int S = a.p.stages;
  const uint32_t ring = smem_u32(smem) + a.p.ring_at + warp * S * a.p.sub_bytes;
  float* sums = reinterpret_cast<float*>(smem + a.p.ring_at);
  const int share = (a.H + gridDim.x - 1) / gridDim.x;
  const int c_begin = min(a.H, (int)blockIdx.x * share), c_end = min(a.H, c_begin + share);
  const int flat = n.units * rs.steps + (shared ? ss.steps : 0);
  const int f0 = (int)((int64_t)flat * warp / kFewWarps);
  const int f1 = (int)((int64_t)flat * (warp + 1) / kFewWarps);
  const uint32_t es = a.scale_dtype == MOE_DT_FP32 ? 4 : 2;
  bool waited = false;

  for (int c0 = c_begin; c0 < c_end; c0 += 16 * kFewDownTiles) {
    const int channels = min(c_end - c0, 16 * kFewDownTiles);
    const int tiles = (channels + 15) / 16;
    auto unit_at = [&](int f, int* u, int* step) {
      if (f < n.units * rs.steps) {
        *u = f / rs.steps;
        *step = f % rs.steps;
      } else {
        *u = n.units;
        *step = f - n.units * rs.steps;
      }
    };
    int next_f = f0, next_m = 0;
    uint32_t fill = 0, use = 0;
    auto issue = [&]() {
      if (next_f < f1) {
        int u, step;
        unit_at(next_f, &u, &step);
        const int e = units[u].expert;
        const FewMatrix& m = e < 0 ? a.shared[2] : a.m[2];
        const FewShape& sh = e < 0 ? ss : rs;
        const int64_t first = e < 0 ? 0 : (int64_t)e * a.H;
        auto row = [&](int r) { return first + min(c0 + next_m * 16 + r, c_end - 1); };
        const unsigned char* wp[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) wp[i] = m.w + row(lane / 8 + 4 * i) * sh.row;
        const unsigned char *sp = nullptr, *zp = nullptr;
        if constexpr (K::kFour) {
          sp = m.s + row(lane / 2) * sh.groups * es;
          if constexpr (K::kZeros) zp = m.z + row(lane / 2) * sh.groups;
        }
        const unsigned char* const wc[4] = {wp[0], wp[1], wp[2], wp[3]};
        copy_stage<K>(a, sh, ring + fill, step, wc, sp, zp);
        if (++next_m == tiles) {
          next_m = 0;
          ++next_f;
        }
      }
      cp_async_commit();
      fill = fill == (uint32_t)(S - 1) * a.p.sub_bytes ? 0u : fill + a.p.sub_bytes;
    };
    for (int i = 0; i < S - 1; ++i) issue();
    if (!waited) {
      // every tile's h is stored (bounded: a tile belongs to a running team)
      if (tid == 0 && !wait_rows_done(&a.head->done, n.total))
        raise_status(a.status, kStTimeout, MOE_K_FEW_FFN);
      __syncthreads();
      waited = true;
    }

    float acc[kFewDownTiles][4] = {}, total[kFewDownTiles][4] = {};
    int unit = -1;
    float w0 = 0.f, w1 = 0.f, up = 1.f;
    const float* hrow = nullptr;
    auto flush = [&]() {
#pragma unroll
      for (int m = 0; m < kFewDownTiles; ++m) {
        total[m][0] = fmaf(w0, acc[m][0], total[m][0]);
        total[m][1] = fmaf(w1, acc[m][1], total[m][1]);
        total[m][2] = fmaf(w0, acc[m][2], total[m][2]);
        total[m][3] = fmaf(w1, acc[m][3], total[m][3]);
        acc[m][0] = acc[m][1] = acc[m][2] = acc[m][3] = 0.f;
      }
    };
    for (int f = f0; f < f1; ++f) {
      int u, step;
      unit_at(f, &u, &step);
      if (u != unit) {
        if (unit >= 0) flush();
        unit = u;
        const uint32_t tokens = units[u].tokens;
        hrow = g < a.T && ((tokens >> g) & 1u) ? a.h + ((int64_t)u * a.T + g) * a.inter : nullptr;
        w0 = units[u].w[2 * tg];
        w1 = units[u].w[2 * tg + 1];
        if constexpr (K::kScaled) {
          up = __uint_as_float(fp16_range_bits(__ldcg(&a.head->hmax[u][g])));
          w0 *= inverse_pow2(fp16_range_bits(__ldcg(&a.head->hmax[u][2 * tg])));
          w1 *= inverse_pow2(fp16_range_bits(__ldcg(&a.head->hmax[u][2 * tg + 1])));
        }
      }
      const int e = units[u].expert;
      const FewShape& sh = e < 0 ? ss : rs;
      // the lane's h of this step, as MMA operands
      uint32_t b[K::kWords][4], rest[K::kRest ? K::kWords : 1][4];
#pragma unroll
      for (int i = 0; i < K::kWords; ++i) {
        const int k = step * K::kStepK + K::k_of(i, tg);
        float4 p = make_float4(0.f, 0.f, 0.f, 0.f), q = p;
        if (hrow && k < sh.K) {
          p = __ldcg(reinterpret_cast<const float4*>(hrow + k));
          q = __ldcg(reinterpret_cast<const float4*>(hrow + k + 4));
        }
        const float v[8] = {p.x * up, p.y * up, p.z * up, p.w * up,
                            q.x * up, q.y * up, q.z * up, q.w * up};
        if constexpr (K::kFour) {
          K::operands(v, b[i]);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            split2<typename K::Mma>(v[2 * j], v[2 * j + 1], b[i][j], rest[i][j]);
        }
      }
      float2 xs[K::kBlocks];
      if constexpr (K::kFour) {
#pragma unroll
        for (int blk = 0; blk < K::kBlocks; ++blk) {
          float d[4] = {};
#pragma unroll
          for (int i = 0; i < K::kPer; ++i) {
            // ones, and sixteens for what was divided by 16
            mma16816<__half>(d, 0x3c003c00u, 0x3c003c00u, 0x4c004c00u, 0x4c004c00u,
                             b[blk * K::kPer + i][0], b[blk * K::kPer + i][1]);
            mma16816<__half>(d, 0x3c003c00u, 0x3c003c00u, 0x4c004c00u, 0x4c004c00u,
                             b[blk * K::kPer + i][2], b[blk * K::kPer + i][3]);
          }
          xs[blk] = make_float2(d[0], d[1]);
        }
      }
      const int64_t first = (e < 0 ? 0 : (int64_t)e * a.H);
#pragma unroll
      for (int m = 0; m < kFewDownTiles; ++m) {
        if (m >= tiles) break;
        wait_stage(S);
        __syncwarp();
        issue();
        FewSkew skew{};
        if constexpr (K::kFour) {
          const int64_t r0 = first + min(c0 + m * 16 + g, c_end - 1);
          const int64_t r8 = first + min(c0 + m * 16 + g + 8, c_end - 1);
          skew.s = (uint32_t)(r0 * sh.groups * es);
          skew.s8 = (uint32_t)(r8 * sh.groups * es);
          skew.z = (uint32_t)(r0 * sh.groups);
          skew.z8 = (uint32_t)(r8 * sh.groups);
        }
        multiply<K>(ring + use, b, rest, xs, true, a, skew, step, acc[m]);
        use = use == (uint32_t)(S - 1) * a.p.sub_bytes ? 0u : use + a.p.sub_bytes;
      }
    }
    if (unit >= 0) flush();
    cp_async_wait<0>();
    __syncthreads();
    // [warp][channel][token], added in the order of the warps
#pragma unroll
    for (int m = 0; m < kFewDownTiles; ++m) {
      float* r = sums + (warp * 16 * kFewDownTiles + m * 16 + g) * 8 + 2 * tg;
      *reinterpret_cast<float2*>(r) = make_float2(total[m][0], total[m][1]);
      *reinterpret_cast<float2*>(r + 64) = make_float2(total[m][2], total[m][3]);
    }
    __syncthreads();
    for (int i = tid; i < channels * a.T; i += kFewThreads) {
      const int t = i / channels, c = i % channels;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kFewWarps; ++w) v += sums[(w * 16 * kFewDownTiles + c) * 8 + t];
      const int64_t at = c0 + c;
      const float zw = zero_w[t];
      if (zw != 0.f) {
        const uint16_t x = static_cast<const uint16_t*>(a.x)[t * a.ldx + at];
        v = fmaf(zw, a.fp16 ? __half2float(__ushort_as_half(x)) : bf16_to_f(x), v);
      }
      if (a.fp16)
        static_cast<__half*>(a.out)[t * a.ldo + at] = from_f<__half>(v);
      else
        static_cast<__nv_bfloat16*>(a.out)[t * a.ldo + at] = from_f<__nv_bfloat16>(v);
    }
    __syncthreads();
  }
}

// x into shared memory as MMA operands.  Four bits: scaled to fp16's range, its block
// sums and the tokens' inverse scales beside it.
template <typename K>
__device__ __forceinline__ void stage_x(const FewArgs& a, unsigned char* smem, float* x_inverse) {
  const int tid = threadIdx.x, lane = tid % 32;
  const int pieces = (a.H + K::kStepK - 1) / K::kStepK * (K::kStepK / 8);
  __shared__ uint32_t most[kFewMaxT];
  if constexpr (K::kFour) {
    if (tid < kFewMaxT) most[tid] = 0u;
    __syncthreads();
    for (int t = 0; t < a.T; ++t) {
      float m = 0.f;
      for (int j = tid; j < a.H / 8; j += kFewThreads) {
        const uint4 q = load_x8(a.x, t * a.ldx + 8 * j, a.vec);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 v = unpack_x(w[i], a.fp16);
          // a NaN's bits are above every number's
          m = __uint_as_float(max(__float_as_uint(m), max(__float_as_uint(fabsf(v.x)),
                                                          __float_as_uint(fabsf(v.y)))));
        }
      }
      uint32_t bits = __float_as_uint(m);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) bits = max(bits, __shfl_xor_sync(0xffffffffu, bits, o));
      if (lane == 0) atomicMax(&most[t], bits);
    }
    __syncthreads();
    if (tid < kFewMaxT) x_inverse[tid] = inverse_pow2(fp16_range_bits(most[tid]));
  }
  for (int i = tid; i < a.T * pieces; i += kFewThreads) {
    const int t = i / pieces, j = i % pieces;
    uint4 q = make_uint4(0u, 0u, 0u, 0u);
    if (8 * j < a.H) {
      q = load_x8(a.x, t * a.ldx + 8 * j, a.vec);
      if constexpr (K::kFour) {
        const float up = __uint_as_float(fp16_range_bits(most[t]));
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
        float v[8];
#pragma unroll
        for (int l = 0; l < 4; ++l) {
          const float2 f = unpack_x(w[l], a.fp16);
          v[2 * l] = f.x * up;
          v[2 * l + 1] = f.y * up;
        }
        uint32_t b[4];
        K::operands(v, b);
        q = make_uint4(b[0], b[1], b[2], b[3]);
      }
    }
    const int step = j / (K::kStepK / 8);
    *reinterpret_cast<uint4*>(smem + t * a.p.xpitch +
                              (step * (K::kStepK / 8) + K::piece_of_k8(j % (K::kStepK / 8))) * 16) =
        q;
  }
  __syncthreads();
  if constexpr (K::kFour) {
    // sums of what the MMAs multiply
    float* sums = reinterpret_cast<float*>(smem + a.p.sum_at);
    constexpr int kPieces = K::kBlock / 8;
    for (int i = tid; i < pieces / kPieces * kFewMaxT; i += kFewThreads) {
      const int t = i % kFewMaxT, blk = i / kFewMaxT;
      float s = 0.f, s16 = 0.f;
      for (int j = 0; j < kPieces && t < a.T; ++j) {
        const uint4 q =
            *reinterpret_cast<const uint4*>(smem + t * a.p.xpitch + (blk * kPieces + j) * 16);
        const float2 b0 = unpack2<__half>(q.x), b1 = unpack2<__half>(q.y);
        const float2 b2 = unpack2<__half>(q.z), b3 = unpack2<__half>(q.w);
        s += (b0.x + b0.y) + (b2.x + b2.y);
        s16 += (b1.x + b1.y) + (b3.x + b3.y);
      }
      sums[i] = fmaf(16.f, s16, s);
    }
    __syncthreads();
  }
}

template <typename K, int MT>
__global__ void __launch_bounds__(kFewThreads, 1) few_ffn_kernel(const __grid_constant__ FewArgs a) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ float x_inverse[kFewMaxT], zero_w[kFewMaxT];
  const int tid = threadIdx.x;
  // x is complete: the routing kernel let this one start only after its own wait for
  // everything before it.  What the routing kernel writes is read after the wait here.
  stage_x<K>(a, smem, x_inverse);
  pdl_wait();
  FewUnit* units = reinterpret_cast<FewUnit*>(smem + a.p.unit_at);
  const bool shared = a.Is > 0;
  FewTiles n;
  n.units = __ldcg(&a.head->units);
  n.routed = (a.I + 8 * MT - 1) / (8 * MT);
  n.shared = shared ? (a.Is + 8 * MT - 1) / (8 * MT) : 0;
  n.total = n.units * n.routed + n.shared;
  for (int i = tid; i < (n.units + shared) * (kFewUnitBytes / 4); i += kFewThreads)
    reinterpret_cast<uint32_t*>(units)[i] = __ldcg(reinterpret_cast<const uint32_t*>(a.head->unit) + i);
  if (tid < kFewMaxT) zero_w[tid] = __ldcg(&a.head->zero_w[tid]);
  __syncthreads();
  gate_up<K, MT>(a, smem, units, n, x_inverse);
  __syncthreads();
  pdl_trigger();
  down<K>(a, smem, units, n, shared, zero_w);
}

// ------------------------------------------------------------------ launch --
template <int TT>
void launch_route(const Launch& L, const RouteArgs& r) {
  const int E = r.tk.E;
  const size_t need = std::max<size_t>((size_t)TT * r.H * 2,
                                       r.tk.T * E * 16 <= kRouteScratch ? (size_t)r.tk.T * E * 16 : 0);
  set_smem_attr_once(reinterpret_cast<const void*>(few_route_kernel<TT>),
                     kRouteSmem,
                     kAttrFewRoute + (TT == 1 ? 0 : TT == 2 ? 1 : TT == 4 ? 2 : 3));
  launch_begin(L, MOE_K_FEW_ROUTE);
  launch_kernel(few_route_kernel<TT>, dim3(std::min(E, L.num_sms)), dim3(kRouteThreads), need,
                L.stream, r);
  launch_end(L, MOE_K_FEW_ROUTE);
}

template <typename K, int MT>
void launch_ffn_as(const Launch& L, const FewArgs& a, int slot) {
  set_smem_attr_once(reinterpret_cast<const void*>(few_ffn_kernel<K, MT>), kFewSmem,
                     kAttrFewFfn + 2 * slot + MT - 1);
  launch_begin(L, MOE_K_FEW_FFN);
  launch_kernel(few_ffn_kernel<K, MT>, dim3(L.num_sms), dim3(kFewThreads), a.p.bytes, L.stream, a);
  launch_end(L, MOE_K_FEW_FFN);
}
template <typename K>
void launch_ffn(const Launch& L, const FewArgs& a, int mt, int slot) {
  if (mt == 1)
    launch_ffn_as<K, 1>(L, a, slot);
  else
    launch_ffn_as<K, 2>(L, a, slot);
}

struct FewLayout {
  size_t head, logits, scratch, h, total;
};
FewLayout few_layout(const moe_config& c, int T) {
  const int E = c.n_routed + c.n_zero;
  const int units = std::min(c.n_routed, T * c.top_k) + (c.shared_inter > 0);
  FewLayout l;
  auto up = [](size_t v) { return (v + 255) & ~(size_t)255; };
  l.head = 256;
  l.logits = l.head + up(sizeof(FewHead));
  l.scratch = l.logits + up((size_t)T * E * 4);
  l.h = l.scratch + up(T * E * 16 <= kRouteScratch ? 0 : (size_t)T * E * 12);
  l.total = l.h + up((size_t)units * T * std::max(c.inter, c.shared_inter) * 4);
  return l;
}

// Gate/up tiles of 8 channels where few tokens leave few tiles; of 16, which read x
// once for twice the weights, otherwise.
int few_tiles(int T) { return T <= 2 ? 1 : 2; }

moe_status check_few(const moe_config* c, int T) {
  // the layer's own checks of the description; the batch's limits are this file's
  size_t bytes;
  const moe_status s = moe_workspace_size(c, T < 0 ? T : std::min(T, 1), &bytes);
  if (s != MOE_OK) return s;
  if (c->wdtype != MOE_W_BF16) return MOE_ERR_UNSUPPORTED;
  if (T > kFewMaxT || (int64_t)T * c->hidden > kFewMaxTH) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_few_tokens_workspace_size(const moe_config* cfg, int32_t T,
                                                    size_t* bytes) {
  const moe_status s = check_few(cfg, T);
  if (s != MOE_OK) return s;
  if (!bytes) return MOE_ERR_INVALID_ARG;
  *bytes = few_layout(*cfg, T).total;
  return MOE_OK;
}

extern "C" moe_status moe_few_tokens(const moe_config* cfg, const moe_few_weights* wt, int32_t T,
                                     int32_t dtype, const void* x, int64_t ldx,
                                     const float* w_router, const float* bias, int32_t* topk_ids,
                                     float* topk_w, void* out, int64_t ldo, void* ws,
                                     size_t ws_bytes, moe_stream_t stream) {
  const moe_status cs = check_few(cfg, T);
  if (cs != MOE_OK) return cs;
  const moe_config& c = *cfg;
  if (!wt || (dtype != MOE_DT_BF16 && dtype != MOE_DT_FP16)) return MOE_ERR_INVALID_ARG;
  const bool any = c.n_routed > 0 || c.shared_inter > 0;  // weights at all
  const bool four = any && wt->w_dtype == MOE_DT_U4;
  if (any && !four && wt->w_dtype != dtype) return MOE_ERR_INVALID_ARG;
  bool aligned_s = true, aligned_z = true, zeros = false;
  if (four) {
    const int group = wt->group;
    if (group != 0 && group != 32 && group != 64 && group != 128) return MOE_ERR_INVALID_ARG;
    if (wt->scale_dtype < MOE_DT_BF16 || wt->scale_dtype > MOE_DT_FP32) return MOE_ERR_INVALID_ARG;
    const int es = wt->scale_dtype == MOE_DT_FP32 ? 4 : 2;
    for (int i = 0; i < 3; ++i) {
      const int k = i == 0 ? c.hidden : i == 1 ? (c.n_routed ? c.inter : 0) : c.shared_inter;
      if (k % 32 || (group > 0 && k % group)) return MOE_ERR_INVALID_ARG;
      const int groups = group > 0 ? k / group : 1;
      aligned_s = aligned_s && (k == 0 || groups * es % 4 == 0);
      aligned_z = aligned_z && (k == 0 || groups % 4 == 0);
    }
  }
  const moe_few_expert* part[2] = {&wt->routed, &wt->shared};
  for (int i = 0; i < 2; ++i) {
    if (i == 0 ? c.n_routed == 0 : c.shared_inter == 0) continue;
    const moe_few_expert& e = *part[i];
    for (int m = 0; m < 3; ++m) {
      if (T > 0 && (!e.w[m] || (four && !e.scales[m]))) return MOE_ERR_INVALID_ARG;
      if (misaligned16(e.w[m], e.scales[m], e.zeros[m])) return MOE_ERR_ALIGNMENT;
      if (!four && (e.scales[m] || e.zeros[m])) return MOE_ERR_INVALID_ARG;
      // zero points for all matrices or for none
      const bool z = e.zeros[m] != nullptr;
      if (i == 0 && m == 0) zeros = z;
      if (i == 1 && m == 0 && c.n_routed == 0) zeros = z;
      if (T > 0 && z != zeros) return MOE_ERR_INVALID_ARG;
    }
  }
  if (T == 0) return MOE_OK;
  if (!x || !w_router || !out || !ws || ldx < c.hidden || ldo < c.hidden)
    return MOE_ERR_INVALID_ARG;
  if (c.bias_mode != MOE_BIAS_NONE && !bias) return MOE_ERR_INVALID_ARG;
  if (misaligned16(x, w_router, bias, topk_ids, topk_w, out) ||
      (reinterpret_cast<uintptr_t>(ws) & 255u))
    return MOE_ERR_ALIGNMENT;
  const FewLayout l = few_layout(c, T);
  if (ws_bytes < l.total) return MOE_ERR_WORKSPACE_TOO_SMALL;

  FewArgs a{};
  const int units = std::min(c.n_routed, T * c.top_k) + (c.shared_inter > 0);
  int mt = few_tiles(T);
  const int es = wt->scale_dtype == MOE_DT_FP32 ? 4 : 2;
  a.p = few_plan(T, c.hidden, units, four, wt->group, es, zeros, aligned_s, aligned_z, mt);
  if (a.p.stages < 3 && mt > 1)
    a.p = few_plan(T, c.hidden, units, four, wt->group, es, zeros, aligned_s, aligned_z, mt = 1);
  if (a.p.stages < 2) return MOE_ERR_UNSUPPORTED;
  Launch L;
  const moe_status s = open_launch(stream, &L);
  if (s != MOE_OK) return s;
  unsigned char* base = static_cast<unsigned char*>(ws);
  L.status = reinterpret_cast<DevStatus*>(base);

  RouteArgs r{};
  r.tk = topk_args(L, c, T, nullptr, bias, nullptr, nullptr);
  r.x = x;
  r.ldx = ldx;
  r.w_r = w_router;
  r.logits = reinterpret_cast<float*>(base + l.logits);
  r.scratch = reinterpret_cast<float*>(base + l.scratch);
  r.ids = topk_ids;
  r.w = topk_w;
  r.head = reinterpret_cast<FewHead*>(base + l.head);
  r.H = c.hidden;
  r.E_r = c.n_routed;
  r.shared = c.shared_inter > 0;
  r.fp16 = dtype == MOE_DT_FP16;
  r.vec = ldx % 8 == 0;

  a.x = x;
  a.ldx = ldx;
  a.out = out;
  a.ldo = ldo;
  for (int m = 0; m < 3; ++m) {
    for (int i = 0; i < 2; ++i) {
      FewMatrix& d = i ? a.shared[m] : a.m[m];
      d.w = static_cast<const unsigned char*>(part[i]->w[m]);
      d.s = static_cast<const unsigned char*>(part[i]->scales[m]);
      d.z = static_cast<const unsigned char*>(part[i]->zeros[m]);
    }
  }
  a.head = r.head;
  a.status = L.status;
  a.h = reinterpret_cast<float*>(base + l.h);
  a.T = T;
  a.H = c.hidden;
  a.I = c.n_routed > 0 ? c.inter : 0;
  a.Is = c.shared_inter;
  a.inter = std::max(c.inter, c.shared_inter);
  a.fp16 = r.fp16;
  a.vec = r.vec;
  a.group = four ? wt->group : 0;
  a.scale_dtype = four ? wt->scale_dtype : MOE_DT_FP32;

  if (T == 1)
    launch_route<1>(L, r);
  else if (T == 2)
    launch_route<2>(L, r);
  else if (T <= 4)
    launch_route<4>(L, r);
  else
    launch_route<8>(L, r);
  if (!four) {
    if (a.fp16)
      launch_ffn<Sixteen<__half>>(L, a, mt, 0);
    else
      launch_ffn<Sixteen<__nv_bfloat16>>(L, a, mt, 1);
  } else if (a.p.block == 32) {
    zeros ? launch_ffn<Four<32, true>>(L, a, mt, 2) : launch_ffn<Four<32, false>>(L, a, mt, 3);
  } else if (a.p.block == 64) {
    zeros ? launch_ffn<Four<64, true>>(L, a, mt, 4) : launch_ffn<Four<64, false>>(L, a, mt, 5);
  } else {
    zeros ? launch_ffn<Four<128, true>>(L, a, mt, 6) : launch_ffn<Four<128, false>>(L, a, mt, 7);
  }
  return launch_status_take();
}
