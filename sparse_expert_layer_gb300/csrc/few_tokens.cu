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
// 8 channels of an expert (8 gate and 8 up rows, one MMA tile), a quarter of K a warp;
// their parts are added in order, SwiGLU gives h in fp32.  Down: a CTA owns a
// range of output channels of all experts; its 16 warps split the (expert, K) steps
// evenly, apply the routing weights to their own sums, and add them in order: one
// rounded store, no atomics, the same bits on every call.  Between the two a CTA waits
// until all tiles have stored h.  Tiles are claimed, so a tile that a waiting CTA needs
// belongs to a running team, whatever else occupies the GPU; and the first stages of
// the down weights are on their way during the wait.  Every warp streams its weights
// through a cp.async ring of its own, so nothing but a tile's sum needs a barrier.
//
// Measured on a GB300, cold (the weights at 6.78 TB/s): one token through 8 of 256 4-bit experts
// and a shared one, 7168 and 2048 channels, groups of 128: 59 us (31); eight tokens through 64
// bf16 experts, 5120 and 1536 channels: 330 (311); five tokens in fp16, groups of 32 with zero points,
// 2304 and 736 channels: 58 (8.4).  By time stamps, with which the 59 are 66: router, picks and the
// start of the second kernel 13, gate and up 28, the wait for the last CTA 4, h 2, down 16, its sums
// 3.  The bf16 layer waits for memory, the 4-bit ones for the latency of short tiles (three to seven
// steps a warp) at 42% issue.
//
// 4-bit weights: a nibble alone in the low bits of a half is the fp16 subnormal
// q * 2^-24 (four bits up: q * 2^-20, its x is divided by 16), so a weight costs part of
// one AND.  x (and h) are scaled by a power of two for each token that brings their
// largest value to 2^13, which makes them fp16 exactly (bf16 values: down to 2^-26 of
// the largest).  A block's MMAs start from -z times its sum of x (of h: another MMA gives it), so
// they hold 2^-24 times the sum of (q - z) x; scales are applied in fp32.  16-bit weights: x as it
// is.
//
// An MMA cuts off what it adds at 2^-25 of the largest addend, for which a subnormal counts as 2^-14,
// the smallest normal number: at 2^-15 of the largest x of sixteen where that meets q * 2^-24.  h is
// about 1e-6 off by that, 1 to 2e-5 beside channels a thousand times as loud.  With codes brought
// to q * 2^-18 (three shifts more for eight of them) it was 2 to 4e-7 off, which no output showed,
// and one token took 4% longer.
//
// With 16-bit weights h is a sum of two 16-bit numbers, the second of which has MMAs of its own.
// With 4-bit ones, whose products are bound by issue and registers, h is one fp16 number where outputs
// are bf16: these are 1.65e-3 off by their rounding, its 11 bits do not show.  fp16 outputs, 2.1e-4
// off by theirs, were 2.8 to 3.2e-4 off with it, so there a token's h takes two columns of the MMAs,
// for its two terms: four tokens fill them, and an expert with more goes through the down projection
// twice.  That makes calls 5 to 9% longer.
#include <math.h>

#include "few_plan.h"
#include "mma.cuh"
#include "topk.cuh"

namespace moe {

namespace {

constexpr int kFewThreads = 32 * kFewWarps;
constexpr int kRouteThreads = 512;
constexpr int kRouteWarps = kRouteThreads / 32;
constexpr int kFewMaxPicks = kFewMaxT * 32;
constexpr int kFewMaxTH = 65536;           // tokens x hidden
constexpr int kFewMaxInter = 1 << 20;      // rows and tiles are counted in 32 bits
constexpr int kRouteScratch = 96 * 1024;   // top-k scratch in shared memory, at most
// MMAs cut their sums off where fp32 ends, each time the same way: with 16-bit weights what
// sixteen of them hold is added, rounded, to the sum.  (4-bit ones: a block's are scaled and added.)
constexpr int kFewChain = 16;

// One expert with rows (expert -1: the shared one).
struct FewUnit {
  int expert;
  uint32_t tokens;  // bit t: token t picked it
};
static_assert(sizeof(FewUnit) == kFewUnitBytes, "the plan's size");
// Tokens of a unit that the down projection takes at once: as many as the MMAs' eight columns hold,
// kFewPairs where a token's h takes two of them.  That list lies over the gate/up tiles' parts.
struct FewPass {
  int unit;
  uint32_t tokens;
};
constexpr int kFewPairs = kFewMaxT / 2;
static_assert((kFewMaxPicks + 1 + (kFewMaxPicks + kFewMaxT) / (kFewPairs + 1)) * sizeof(FewPass) <=
                  kFewParts,
              "every unit's passes");

// Workspace after the status block.  `ticket` is zero between calls; the rest is
// written by the first kernel.
struct FewHead {
  int ticket;
  int claim, done;  // gate/up tiles claimed and stored
  int units;        // without the shared one
  float zero_w[kFewMaxT];  // weights of the tokens' zero-computation picks
  FewUnit unit[kFewMaxPicks + 1];
  float w[kFewMaxPicks + 1][kFewMaxT];        // a unit's routing weights, 0 for other tokens
  uint32_t hmax[kFewMaxPicks + 1][kFewMaxT];  // largest finite |h| of a unit's token, fp32 bits
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
  int zstep;  // groups of a row in a stage, 0 where a row has one
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
// Top-k without groups in registers; other kinds by topk_token, whose logits and scratch (4 E
// floats a token) lie in shared memory where they fit.
__host__ __device__ inline bool route_flat(const TopkArgs& a) {
  return a.n_group <= 1 && a.E <= 1024;
}
__host__ __device__ inline bool route_scratch_inside(const TopkArgs& a) {
  return !route_flat(a) && a.T * a.E * 16 <= kRouteScratch;
}
__device__ __forceinline__ float2 unpack_x(uint32_t w, int fp16) {
  return fp16 ? unpack2<__half>(w) : unpack2<__nv_bfloat16>(w);
}
// Four, eight channels of a 16-bit row.
__device__ __forceinline__ uint2 load_x4(const void* x, int64_t at, bool vec) {
  const uint16_t* p = static_cast<const uint16_t*>(x) + at;
  if (vec) return *reinterpret_cast<const uint2*>(p);
  return make_uint2(p[0] | (uint32_t)p[1] << 16, p[2] | (uint32_t)p[3] << 16);
}
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

// The sums of N values over the warp, N a power of two up to 32: lane i * 32 / N (and the
// lanes that follow it, up to the next one) ends up with that of v[i].
template <int N>
__device__ __forceinline__ float warp_sums(float (&v)[N]) {
  const int lane = threadIdx.x % 32;
  int o = 16;
#pragma unroll
  for (int n = N / 2; n > 0; n /= 2, o /= 2) {
    const bool upper = lane & o;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float mine = upper ? v[i + n] : v[i], theirs = upper ? v[i] : v[i + n];
      v[i] = mine + __shfl_xor_sync(0xffffffffu, theirs, o);
    }
  }
  float s = v[0];
  for (; o > 0; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// Larger floats are larger numbers; what can not be picked (-inf, NaN) is 0.
__device__ __forceinline__ uint32_t pick_key(float v) {
  const uint32_t b = __float_as_uint(v);
  return v > -INFINITY ? b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u) : 0u;
}

// topk_token (topk.cuh) without groups for at most 32 * N experts: a lane keeps those of every
// 32nd expert in registers, a pick is a maximum over the warp by redux.  The same scores, order
// and weights.
template <int N>
__device__ __forceinline__ void pick_flat(const TopkArgs& a, int t, const float* row) {
  const int lane = threadIdx.x % 32;
  float score[N], bias[N];
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = lane + 32 * i;
    score[i] = e < a.E ? __ldcg(row + e) : -INFINITY;
    bias[i] = e < a.E && a.bias_mode != MOE_BIAS_NONE ? a.bias[e] : 0.f;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (a.bias_mode == MOE_BIAS_LOGIT) score[i] += bias[i];
    m = fmaxf(m, score[i]);
  }
  if (a.score == MOE_SCORE_SOFTMAX) {
    m = warp_max(m);
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      score[i] = lane + 32 * i < a.E ? expf(score[i] - m) : 0.f;
      z += score[i];
    }
    z = warp_sum(z);
#pragma unroll
    for (int i = 0; i < N; ++i) score[i] = score[i] / z;
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) score[i] = 1.f / (1.f + expf(-score[i]));
  }
  uint32_t key[N];
#pragma unroll
  for (int i = 0; i < N; ++i)
    key[i] = lane + 32 * i >= a.E                ? 0u
             : a.bias_mode == MOE_BIAS_SELECT ? pick_key(score[i] + bias[i])
                                              : pick_key(score[i]);
  int my_id = 0;
  float my_w = 0.f;
  for (int j = 0; j < a.k; ++j) {
    uint32_t best = 0u;
    int at = 0;
    float w = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (key[i] > best) {
        best = key[i];
        at = i;
        w = score[i];
      }
    const uint32_t top = __reduce_max_sync(0xffffffffu, best);
    const uint32_t mine = best == top ? (uint32_t)(lane + 32 * at) : 0xffffffffu;
    uint32_t id = __reduce_min_sync(0xffffffffu, mine);
    if (top == 0u) {  // fewer eligible experts than k (non-finite keys)
      if (lane == 0) raise_status(a.status, kStInternal, MOE_K_FEW_ROUTE);
      id = 0u;
      w = score[0];
    }
    w = __shfl_sync(0xffffffffu, w, id % 32);
    if (lane == j) {
      my_id = (int)id;
      my_w = w;
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (id == (uint32_t)(lane + 32 * i)) key[i] = 0u;
  }
  const float sum = warp_sum(lane < a.k ? my_w : 0.f);
  if (lane < a.k) {
    a.ids[t * a.k + lane] = my_id;
    a.w[t * a.k + lane] = (a.renorm ? my_w / sum : my_w) * a.scale;
  }
}

// Logits of the CTA's experts for all TT >= T tokens; the last CTA picks.  A thread keeps its
// columns of all tokens in registers and meets two rows of W_r at a time with them; the first
// rows are on their way while x arrives.
template <int TT>
__global__ void __launch_bounds__(kRouteThreads) few_route_kernel(RouteArgs a) {
  pdl_enter();
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ float part[kRouteWarps][2 * TT];
  __shared__ int32_t ids[kFewMaxPicks];
  __shared__ float wts[kFewMaxPicks];
  __shared__ bool first[kFewMaxPicks];
  __shared__ int last;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int T = a.tk.T, H = a.H, E = a.tk.E, k = a.tk.k, G = gridDim.x;
  constexpr int kCols = 4;  // float4 of a row that a thread holds at once
  constexpr int kSpan = kCols * kRouteThreads;
  for (int r = blockIdx.x; r < E; r += 2 * G) {
    const bool two = r + G < E;
    const float4* w0 = reinterpret_cast<const float4*>(a.w_r + (size_t)r * H);
    const float4* w1 = reinterpret_cast<const float4*>(a.w_r + (size_t)(two ? r + G : r) * H);
    float acc[2 * TT] = {};
    for (int c0 = tid; c0 - tid < H / 4; c0 += kSpan) {
      float4 v0[kCols], v1[kCols];
#pragma unroll
      for (int i = 0; i < kCols; ++i) {
        const int c = c0 + i * kRouteThreads;
        const bool in = c < H / 4;
        v0[i] = in ? __ldg(w0 + c) : make_float4(0.f, 0.f, 0.f, 0.f);
        v1[i] = in && two ? __ldg(w1 + c) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      uint2 x[TT][kCols];
#pragma unroll
      for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int i = 0; i < kCols; ++i) {
          const int c = c0 + i * kRouteThreads;
          x[t][i] = t < T && c < H / 4 ? load_x4(a.x, t * a.ldx + 4 * c, a.vec) : make_uint2(0u, 0u);
        }
#pragma unroll
      for (int i = 0; i < kCols; ++i)
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          const float2 x0 = unpack_x(x[t][i].x, a.fp16), x1 = unpack_x(x[t][i].y, a.fp16);
          acc[t] = fmaf(v0[i].x, x0.x, acc[t]);
          acc[t] = fmaf(v0[i].y, x0.y, acc[t]);
          acc[t] = fmaf(v0[i].z, x1.x, acc[t]);
          acc[t] = fmaf(v0[i].w, x1.y, acc[t]);
          acc[TT + t] = fmaf(v1[i].x, x0.x, acc[TT + t]);
          acc[TT + t] = fmaf(v1[i].y, x0.y, acc[TT + t]);
          acc[TT + t] = fmaf(v1[i].z, x1.x, acc[TT + t]);
          acc[TT + t] = fmaf(v1[i].w, x1.y, acc[TT + t]);
        }
    }
    const float s = warp_sums<2 * TT>(acc);
    constexpr int kEach = 32 / (2 * TT);  // lanes with the same sum
    if (lane % kEach == 0) part[warp][lane / kEach] = s;
    __syncthreads();
    if (tid < 2 * TT) {
      const int j = tid / TT, t = tid % TT;
      float v = 0.f;
#pragma unroll
      for (int i = 0; i < kRouteWarps; ++i) v += part[i][tid];
      if (t < T && (j == 0 || two)) a.logits[(size_t)t * E + r + j * G] = v;
    }
    __syncthreads();
  }
  if (warp == 0) {  // (the warp that stored the logits)
    __syncwarp();
    if (lane == 0) {
      __threadfence();
      last = atomicAdd(&a.head->ticket, 1) == G - 1;
      __threadfence();
    }
  }
  __syncthreads();
  if (!last) return;

  // Picks of all tokens, a warp each.
  const bool flat = route_flat(a.tk), inside = route_scratch_inside(a.tk);
  float* lg = reinterpret_cast<float*>(smem);
  for (int i = tid; i < T * E && inside; i += kRouteThreads) lg[i] = __ldcg(a.logits + i);
  if (inside) __syncthreads();
  if (warp < T) {
    TopkArgs tk = a.tk;
    tk.ids = ids;
    tk.w = wts;
    const float* row = inside ? lg + warp * E : a.logits + (size_t)warp * E;
    if (!flat)
      topk_token(tk, warp, row,
                 inside ? lg + T * E + warp * 3 * E : a.scratch + (size_t)warp * 3 * E);
    else if (E <= 256)
      pick_flat<8>(tk, warp, row);
    else if (E <= 512)
      pick_flat<16>(tk, warp, row);
    else if (E <= 768)
      pick_flat<24>(tk, warp, row);
    else
      pick_flat<32>(tk, warp, row);
  }
  __syncthreads();

  // Units: the distinct experts with weights, in order of their first pick; a warp a pick,
  // lanes compare it with the others.
  FewHead* head = a.head;
  const int picks = T * k;
  for (int p = warp; p < picks; p += kRouteWarps) {
    const int e = ids[p];
    bool earlier = e < 0 || e >= a.E_r;
    for (int i = lane; i < p; i += 32) earlier = earlier || ids[i] == e;
    earlier = __any_sync(0xffffffffu, earlier);
    if (lane == 0) first[p] = !earlier;
  }
  __syncthreads();
  int units = 0;
  for (int i0 = 0; i0 < picks; i0 += 32)
    units += __popc(__ballot_sync(0xffffffffu, i0 + lane < picks && first[i0 + lane]));
  for (int p = warp; p < picks; p += kRouteWarps) {
    if (!first[p]) continue;
    const int e = ids[p];
    int at = 0;
    for (int i0 = 0; i0 < p; i0 += 32)
      at += __popc(__ballot_sync(0xffffffffu, i0 + lane < p && first[i0 + lane]));
    uint32_t tokens = 0u;
    if (lane < kFewMaxT) head->w[at][lane] = 0.f;
    __syncwarp();
    for (int i = p + lane; i < picks; i += 32)
      if (ids[i] == e) {
        tokens |= 1u << (i / k);
        head->w[at][i / k] = wts[i];
      }
    tokens = __reduce_or_sync(0xffffffffu, tokens);
    if (lane == 0) head->unit[at] = {e, tokens};
  }
  if (tid < kFewMaxT) {
    float z = 0.f;
    for (int j = 0; j < k && tid < T; ++j)
      if (ids[tid * k + j] >= a.E_r) z += wts[tid * k + j];
    head->zero_w[tid] = z;
  }
  if (tid == 0) {
    if (a.shared) {
      head->unit[units] = {-1, (1u << T) - 1u};
#pragma unroll
      for (int t = 0; t < kFewMaxT; ++t) head->w[units][t] = t < T ? 1.f : 0.f;
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
// 16 bytes of a weight row.  Past its end (in false) codes are left as they are: whatever
// lies there is finite and meets zeros of x; 16-bit weights become zeros (src is not read).
// Weights leave L2 first: they pass once, and what stays is the kernel's own instructions and h.
template <bool FOUR>
__device__ __forceinline__ void copy_piece(uint32_t dst, const unsigned char* src, bool in,
                                           const void* safe, uint64_t policy) {
  if constexpr (FOUR) {
    if (in)
      asm volatile("cp.async.cg.shared.global.L2::cache_hint.L2::256B [%0], [%1], 16, %2;" ::"r"(dst),
                   "l"(src), "l"(policy)
                   : "memory");
  } else {
    asm volatile("cp.async.cg.shared.global.L2::cache_hint.L2::256B [%0], [%1], 16, %2, %3;" ::"r"(dst),
                 "l"(in ? static_cast<const void*>(src) : safe), "r"(in ? 16 : 0), "l"(policy)
                 : "memory");
  }
}
__device__ __forceinline__ void team_barrier(int team) {
  asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "n"(32 * kFewTeamWarps) : "memory");
}
// All but the `stages - 2` groups committed last have arrived.
__device__ __forceinline__ void wait_stage(int stages) {
  if (stages == 4)
    cp_async_wait<2>();
  else if (stages == 3)
    cp_async_wait<1>();
  else
    cp_async_wait<0>();
}
static_assert(kFewMaxStages == 4, "wait_stage knows up to four");

template <typename T>
__device__ __forceinline__ float read_scale(uint32_t at) {
  if constexpr (sizeof(T) == 4) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
  } else {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at) : "memory");
    if constexpr (std::is_same<T, __half>::value)
      return __half2float(__ushort_as_half(v));
    else
      return bf16_to_f(v);
  }
}
__device__ __forceinline__ float read_zero(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return (float)(v & 31u);
}
// d = a b + (c0, c1, c2, c3)
__device__ __forceinline__ void mma_from(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1, float c0, float c1,
                                         float c2, float c3) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

// The kinds of weights.  kWords: granules of eight K that a lane supplies in a stage;
// granule i is x's 16-byte piece piece(i, tg) of the stage.
template <int BLOCK, bool ZEROS, typename SCALE, bool PAIRED>
struct Four {
  using Mma = __half;
  using Scale = SCALE;
  static constexpr bool kFour = true, kZeros = ZEROS, kScaled = true;
  // a second term of h has MMAs or columns of its own
  static constexpr bool kRest = false, kPaired = PAIRED, kTwo = PAIRED;
  static constexpr int kStepK = 256, kWords = 8, kScaleBytes = sizeof(SCALE);
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
  static __device__ __forceinline__ void order(float (&v)[8]) {
    const float w[8] = {v[0], v[4], v[1] * 0.0625f, v[5] * 0.0625f,
                        v[2], v[6], v[3] * 0.0625f, v[7] * 0.0625f};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = w[i];
  }
};
template <typename T>
struct Sixteen {
  using Mma = T;
  static constexpr bool kFour = false, kRest = true, kPaired = false, kTwo = true;
  static constexpr bool kScaled = std::is_same<T, __half>::value;  // h needs fp16's range
  static constexpr int kStepK = 64, kWords = 2, kBlocks = 1;
  static __device__ __forceinline__ int k_of(int i, int tg) { return i * 32 + tg * 8; }
  static __device__ __forceinline__ int piece(int i, int tg) { return i * 4 + tg; }
  static __device__ __forceinline__ int piece_of_k8(int j) { return j; }
  static __device__ __forceinline__ int swizzle(int r, int c) { return c ^ ((r & 1) << 2); }
};

// Where a lane finds the groups of its row g in a stage (row g + 8: `eight` bytes on; the
// byte inside the first word is the same there).
struct FewGroups {
  uint32_t s;  // scales
  uint32_t z;  // zero points, less the byte inside their first word
  uint32_t zbyte;
};

// acc += the sum over a stage's K of its 16 rows times b: 2^-24 of it with 4-bit weights.
// xs: minus 8 x 2^-24 times the sums of x over the stage's blocks (with zero points: minus
// 2^-24 times them), for the lane's columns 2 tg and 2 tg + 1.  row: the stage and the lane's
// row g in it.
template <typename K, bool REST>
__device__ __forceinline__ void multiply(uint32_t st, const uint32_t (&b)[K::kWords][4],
                                         const uint32_t (&rest)[REST ? K::kWords : 1][4],
                                         const float2 (&xs)[K::kBlocks], const FewArgs& a,
                                         const FewGroups& at, int step, float (&acc)[4]) {
  const int lane = threadIdx.x % 32, g = lane / 4, tg = lane % 4;
  const uint32_t row = st + g * 128;
  if constexpr (K::kFour) {
    const uint32_t s0 = st + at.s, s8 = s0 + a.p.s_eight;
    uint32_t z0 = 0, z8 = 0;
    if constexpr (K::kZeros) {
      z0 = st + at.z + ((at.zbyte + step * a.zstep) & 3u);
      z8 = z0 + a.p.z_eight;
    }
#pragma unroll
    for (int blk = 0; blk < K::kBlocks; ++blk) {
      uint32_t lo[K::kPer], hi[K::kPer];
      const int byte = blk * (K::kBlock / 2) + tg * (K::kBlock / 8);
      const uint32_t from = row + K::swizzle(g, byte / 16) * 16 + byte % 16;
      if constexpr (K::kPer == 4) {
        const uint4 u = lds128(from), v = lds128(from + 8 * 128);
        lo[0] = u.x, lo[1] = u.y, lo[2] = u.z, lo[3] = u.w;
        hi[0] = v.x, hi[1] = v.y, hi[2] = v.z, hi[3] = v.w;
      } else if constexpr (K::kPer == 2) {
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                     : "=r"(lo[0]), "=r"(lo[1]) : "r"(from) : "memory");
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                     : "=r"(hi[0]), "=r"(hi[1]) : "r"(from + 8 * 128) : "memory");
      } else {
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(lo[0]) : "r"(from) : "memory");
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(hi[0]) : "r"(from + 8 * 128) : "memory");
      }
      // (one scale for the whole row: every block reads the first)
      const uint32_t js = blk * a.p.s_next, jz = blk * a.p.z_next;
      float c0 = xs[blk].x, c1 = xs[blk].y, c2 = c0, c3 = c1;
      if constexpr (K::kZeros) {
        const float za = read_zero(z0 + jz), zb = read_zero(z8 + jz);
        c2 = c0 * zb, c3 = c1 * zb, c0 *= za, c1 *= za;
      }
      const float sa = read_scale<typename K::Scale>(s0 + js);
      const float sb = read_scale<typename K::Scale>(s8 + js);
      float d[4];
#pragma unroll
      for (int i = 0; i < K::kPer; ++i) {
        const int w = blk * K::kPer + i;
        const uint32_t l = lo[i], h = hi[i], l8 = l >> 8, h8 = h >> 8;
        if (i == 0)
          mma_from(d, l & 0x000f000fu, h & 0x000f000fu, l & 0x00f000f0u, h & 0x00f000f0u, b[w][0],
                   b[w][1], c0, c1, c2, c3);
        else
          mma16816<__half>(d, l & 0x000f000fu, h & 0x000f000fu, l & 0x00f000f0u, h & 0x00f000f0u,
                           b[w][0], b[w][1]);
        mma16816<__half>(d, l8 & 0x000f000fu, h8 & 0x000f000fu, l8 & 0x00f000f0u,
                         h8 & 0x00f000f0u, b[w][2], b[w][3]);
      }
      acc[0] = fmaf(sa, d[0], acc[0]);
      acc[1] = fmaf(sa, d[1], acc[1]);
      acc[2] = fmaf(sb, d[2], acc[2]);
      acc[3] = fmaf(sb, d[3], acc[3]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < K::kWords; ++i) {
      const uint32_t from = row + K::swizzle(g, i * 4 + tg) * 16;
      const uint4 u = lds128(from), v = lds128(from + 8 * 128);
      mma16816<typename K::Mma>(acc, u.x, v.x, u.y, v.y, b[i][0], b[i][1]);
      mma16816<typename K::Mma>(acc, u.z, v.z, u.w, v.w, b[i][2], b[i][3]);
      if constexpr (REST) {
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

// The scales and zero points of a stage's row lane / 2, whose groups begin at sp and zp.
// Where all rows are whole stages (a.p.whole) the scales of a stage are one aligned copy (or
// two); otherwise words lane % 2, + 2, .. of each, up to the row's end.
template <typename K>
__device__ __forceinline__ void copy_groups(const FewArgs& a, int groups, uint32_t st, int step,
                                            const unsigned char* sp, const unsigned char* zp) {
  const int lane = threadIdx.x % 32;
  auto words = [&](const unsigned char* row, int first, int end, int n, uint32_t dst) {
    const uint32_t byte = (uint32_t)(reinterpret_cast<uintptr_t>(row + first) & 3u);
    const unsigned char* const first_word = row + first - byte;
    const unsigned char* from = first_word + 4 * (lane % 2);
    int left = end - first + (int)byte - 4 * (lane % 2);
    dst += lane / 2 * 4 * n + 4 * (lane % 2);
    for (int i = lane % 2; i < n; i += 2, from += 8, left -= 8, dst += 8)
      cp_async_word(dst, left > 0 ? from : first_word, max(0, min(4, left)));
  };
  constexpr int kRun = K::kBlocks * K::kScaleBytes;  // of a row
  if (a.p.whole) {
    const unsigned char* from = sp + step * kRun;
    const uint32_t dst = st + kFewSub + lane / 2 * kRun;
    if constexpr (kRun == 32) {
      cp_async16(dst + lane % 2 * 16, from + lane % 2 * 16);
    } else if (lane % 2 == 0) {
      cp_async_unit(dst, from, kRun);
    }
  } else {
    words(sp, step * a.zstep * K::kScaleBytes, groups * K::kScaleBytes, a.p.swords, st + kFewSub);
  }
  if constexpr (K::kZeros) {
    if (a.p.whole && K::kBlocks >= 4) {
      if (lane % 2 == 0)
        cp_async_unit(st + kFewSub + 64 * a.p.swords + lane / 2 * K::kBlocks, zp + step * K::kBlocks,
                      K::kBlocks);
    } else {
      words(zp, step * a.zstep, groups, a.p.zwords, st + kFewSub + 64 * a.p.swords);
    }
  }
}
template <typename K>
__device__ __forceinline__ FewGroups groups_at(const FewArgs& a, const FewShape& sh, int64_t row) {
  const int g = threadIdx.x % 32 / 4;
  FewGroups at{};
  if constexpr (K::kFour) {
    at.s = kFewSub + g * 4 * a.p.swords + ((uint32_t)(row * sh.groups * K::kScaleBytes) & 3u);
    at.z = kFewSub + 64 * a.p.swords + g * 4 * a.p.zwords;
    at.zbyte = (uint32_t)(row * sh.groups);
  }
  return at;
}

// The numbering of the gate/up tiles.
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

template <typename K>
__device__ __forceinline__ void gate_up(const FewArgs& a, unsigned char* smem, const FewUnit* units,
                                        const FewTiles& n, const float* x_inverse) {
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int team = warp / kFewTeamWarps, kw = warp % kFewTeamWarps, tt = tid % (32 * kFewTeamWarps);
  const int g = lane / 4, tg = lane % 4;
  const FewShape sh = shape_of<K>(a, a.H);
  const int per = (sh.steps + kFewTeamWarps - 1) / kFewTeamWarps;
  const int k0 = min(sh.steps, kw * per), k1 = min(sh.steps, k0 + per);
  const int S = a.p.stages, sub = a.p.sub_bytes;
  // tiles a team knows beyond the one it works on: as many as its rings reach into
  const int least = sh.steps - (sh.steps - 1) / per * per;  // the last busy warp's steps
  const int ahead = (S - 1 + least - 1) / least;
  volatile int* queue = reinterpret_cast<int*>(smem + a.p.queue_at) + team * 16;
  float* red = reinterpret_cast<float*>(smem + a.p.red_at) + team * 2 * kFewTeamWarps * 128;
  const uint32_t ring = smem_u32(smem) + a.p.ring_at + warp * S * sub;
  FewHead* head = a.head;
  if (tt == 0) {
    const int base = atomicAdd(&head->claim, ahead + 1);
    for (int i = 0; i <= ahead; ++i) queue[i] = base + i;
  }
  team_barrier(team);

  // What is copied next: the tile of queue[seq], `togo` stages of it.  The lane copies its
  // piece of rows lane / 8 and four on of both matrices, and groups of row lane / 2.
  int seq_next = 0, togo = 0, step_next = 0, left = 0;
  bool done = k0 == k1;
  const unsigned char *gate0 = nullptr, *gate1 = nullptr, *up0 = nullptr, *up1 = nullptr;
  const unsigned char *sp = nullptr, *zp = nullptr;
  const int dst = lane / 8 * 128;
  const uint32_t d0 = dst + K::swizzle(lane / 8, lane % 8) * 16;
  const uint32_t d1 = dst + 4 * 128 + K::swizzle(lane / 8 + 4, lane % 8) * 16;
  const uint32_t ring_last = ring + (S - 1) * sub;
  const uint64_t policy = policy_evict_first();
  auto issue = [&](uint32_t slot) {
    if (togo == 0 && !done) {
      const int tile = queue[seq_next++ % 16];
      done = tile >= n.total;
      if (!done) {
        int u, f;
        tile_at(n, tile, &u, &f);
        const int e = units[u].expert;
        const FewMatrix* m = e < 0 ? a.shared : a.m;
        const int64_t row = (e < 0 ? 0 : (int64_t)e * a.I) + f * 8;
        const int64_t at = (row + lane / 8) * sh.row + k0 * 128 + (lane % 8) * 16;
        gate0 = m[0].w + at;
        gate1 = gate0 + 4 * sh.row;
        up0 = m[1].w + at;
        up1 = up0 + 4 * sh.row;
        left = sh.row - k0 * 128 - (lane % 8) * 16;
        if constexpr (K::kFour) {
          const int64_t first = (row + lane / 2 % 8) * sh.groups;  // rows 0-7 are gate's
          sp = (lane < 16 ? m[0].s : m[1].s) + first * K::kScaleBytes;
          if constexpr (K::kZeros) zp = (lane < 16 ? m[0].z : m[1].z) + first;
        }
        togo = k1 - k0;
        step_next = k0;
      }
    }
    if (togo) {
      const bool in = left > 0;
      copy_piece<K::kFour>(slot + d0, gate0, in, a.x, policy);
      copy_piece<K::kFour>(slot + d1, gate1, in, a.x, policy);
      copy_piece<K::kFour>(slot + d0 + 8 * 128, up0, in, a.x, policy);
      copy_piece<K::kFour>(slot + d1 + 8 * 128, up1, in, a.x, policy);
      if constexpr (K::kFour) copy_groups<K>(a, sh.groups, slot, step_next, sp, zp);
      gate0 += 128;
      gate1 += 128;
      up0 += 128;
      up1 += 128;
      left -= 128;
      ++step_next;
      --togo;
    }
    cp_async_commit();
  };
  for (int i = 0; i < S - 1; ++i) issue(ring + i * sub);

  uint32_t use = ring, before = ring_last;  // the stage to be used, the one used last
  const uint32_t x0 = smem_u32(smem) + min(g, a.T - 1) * a.p.xpitch + tg * 16 +
                      k0 * (K::kStepK * 2);
  const uint32_t sum0 = smem_u32(smem) + a.p.sum_at + tg * 8 + k0 * (K::kBlocks * kFewMaxT * 4);
  int stored = 0;
  for (int seq = 0;; ++seq) {
    const int tile = queue[seq % 16];
    if (tile >= n.total) break;
    int claimed = 0;
    if (tt == 0) claimed = atomicAdd(&head->claim, 1);
    int u, f;
    tile_at(n, tile, &u, &f);
    const int e = units[u].expert;
    const FewGroups at = groups_at<K>(a, sh, (e < 0 ? 0 : (int64_t)e * a.I) + f * 8 + g);
    float acc[4] = {}, sum[4] = {};
    auto flush = [&]() {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sum[i] += acc[i];
        acc[i] = 0.f;
      }
    };
    uint32_t xat = x0, sum_at = sum0;
    for (int step = k0; step < k1; ++step) {
      wait_stage(S);
      __syncwarp();
      issue(before);
      uint32_t b[K::kWords][4];
      float2 xs[K::kBlocks];
#pragma unroll
      for (int i = 0; i < K::kWords; ++i) {
        const uint4 v = lds128(xat + K::piece(i, 0) * 16);
        b[i][0] = v.x, b[i][1] = v.y, b[i][2] = v.z, b[i][3] = v.w;
      }
      xat += K::kStepK * 2;
      if constexpr (K::kFour) {
#pragma unroll
        for (int i = 0; i < K::kBlocks; ++i)
          asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];"
                       : "=f"(xs[i].x), "=f"(xs[i].y)
                       : "r"(sum_at + i * kFewMaxT * 4)
                       : "memory");
        sum_at += K::kBlocks * kFewMaxT * 4;
      }
      const uint32_t none[1][4] = {};
      multiply<K, false>(use, b, none, xs, a, at, step, acc);
      if constexpr (!K::kFour) {
        constexpr int kSteps = kFewChain / (2 * K::kWords);
        if ((step - k0) % kSteps == kSteps - 1) flush();
      }
      before = use;
      use = use == ring_last ? ring : use + sub;
    }
    // The parts meet in one of two buffers; one warp of the team, another each time, adds them
    // and stores h while the others go on.  (The buffer's next use is past the next barrier,
    // which that warp reaches when it is done.)
    flush();
    float* parts = red + (seq & 1) * kFewTeamWarps * 128;
    float* r = parts + kw * 128 + g * 8 + 2 * tg;
    *reinterpret_cast<float2*>(r) = make_float2(sum[0], sum[1]);
    *reinterpret_cast<float2*>(r + 64) = make_float2(sum[2], sum[3]);
    if (tt == 0) queue[(seq + ahead + 1) % 16] = claimed;
    team_barrier(team);
    if (kw == seq % kFewTeamWarps) {
      const int ch = lane % 8;
      const uint32_t tokens = units[u].tokens;
      for (int t = lane / 8; t - lane / 8 < a.T; t += 4) {
        float gate = 0.f, up = 0.f;
#pragma unroll
        for (int i = 0; i < kFewTeamWarps; ++i) {
          gate += parts[i * 128 + ch * 8 + t];
          up += parts[i * 128 + (ch + 8) * 8 + t];
        }
        const bool mine = (tokens >> t) & 1u;
        float h = 0.f;
        if (mine) {
          if constexpr (K::kFour) {
            gate = gate * 16777216.f * x_inverse[t];
            up = up * 16777216.f * x_inverse[t];
          }
          h = gate / (1.f + expf(-gate)) * up;
          __stcg(a.h + ((int64_t)u * a.T + t) * a.inter + f * 8 + ch, h);
        }
        if constexpr (K::kScaled) {
          uint32_t most = magnitude(h);
#pragma unroll
          for (int o = 4; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
          if (ch == 0 && mine) atomicMax(&head->hmax[u][t], most);
        }
      }
    }
    ++stored;
  }
  cp_async_wait<0>();
  // The team's tiles are stored: one fence for all of them (one a tile held up the warp that
  // finished it by a microsecond).
  team_barrier(team);
  if (tt == 0) {
    __threadfence();
    atomicAdd(&head->done, stored);
  }
}

constexpr int kFewDownTiles = 4;  // 16-row tiles of one pass of the down projection

// Eight values of h as MMA operands, scaled by `up`; rest: what 16-bit operands leave of them.
template <typename K>
__device__ __forceinline__ void h_operands(const float4& p, const float4& q, float up,
                                           uint32_t (&b)[4], uint32_t (&rest)[4]) {
  float v[8] = {p.x * up, p.y * up, p.z * up, p.w * up, q.x * up, q.y * up, q.z * up, q.w * up};
  if constexpr (K::kFour) K::order(v);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (K::kTwo)
      split2<typename K::Mma>(v[2 * j], v[2 * j + 1], b[j], rest[j]);
    else
      b[j] = pack2<typename K::Mma>(v[2 * j], v[2 * j + 1]);
  }
}

// All rows of h as operands in shared memory, over x: where they fit, each CTA turns them into
// operands once and not for every tile of channels.  row[r]: unit * 8 + token.
template <typename K>
__device__ __forceinline__ void stage_h(const FewArgs& a, unsigned char* smem,
                                        const FewUnit* units, int rows, const int* row) {
  const int pieces = (a.p.hpitch - 64) / 16, n = rows * pieces;
  constexpr int kAtOnce = 4;
  for (int e0 = threadIdx.x; e0 < n; e0 += kAtOnce * kFewThreads) {
    float4 p[kAtOnce], q[kAtOnce];
    uint32_t most[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int e = e0 + i * kFewThreads, r = e / pieces, j = e % pieces;
      p[i] = q[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      most[i] = 0u;
      if (e >= n) continue;
      const int u = row[r] / kFewMaxT, t = row[r] % kFewMaxT;
      if (8 * j < (units[u].expert < 0 ? a.Is : a.I)) {
        const float* from = a.h + ((int64_t)u * a.T + t) * a.inter + 8 * j;
        p[i] = __ldcg(reinterpret_cast<const float4*>(from));
        q[i] = __ldcg(reinterpret_cast<const float4*>(from + 4));
      }
      if constexpr (K::kScaled) most[i] = __ldcg(&a.head->hmax[u][t]);
    }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int e = e0 + i * kFewThreads, r = e / pieces, j = e % pieces;
      if (e >= n) break;
      const float up = K::kScaled ? __uint_as_float(fp16_range_bits(most[i])) : 1.f;
      uint32_t b[4], rest[4];
      h_operands<K>(p[i], q[i], up, b, rest);
      const int step = j / (K::kStepK / 8);
      unsigned char* to = smem + r * a.p.hpitch +
                          (step * (K::kStepK / 8) + K::piece_of_k8(j % (K::kStepK / 8))) * 16;
      *reinterpret_cast<uint4*>(to) = make_uint4(b[0], b[1], b[2], b[3]);
      if constexpr (K::kTwo)
        *reinterpret_cast<uint4*>(to + a.p.hrest) = make_uint4(rest[0], rest[1], rest[2], rest[3]);
    }
  }
}

template <typename K>
__device__ __forceinline__ void down(const FewArgs& a, unsigned char* smem, const FewUnit* units,
                                     const FewTiles& n, const FewPass* passes, int routed_passes,
                                     int shared_passes, int nunits, const float* zero_w) {
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int g = lane / 4, tg = lane % 4;
  const FewShape rs = shape_of<K>(a, a.I), ss = shape_of<K>(a, a.Is);
  const int S = a.p.stages, sub = a.p.sub_bytes;
  const uint32_t ring = smem_u32(smem) + a.p.ring_at + warp * S * sub;
  const uint32_t ring_last = ring + (S - 1) * sub;
  const uint64_t policy = policy_evict_first();
  float* sums = reinterpret_cast<float*>(smem + a.p.ring_at);
  const int share = (a.H + gridDim.x - 1) / gridDim.x;
  const int c_begin = min(a.H, (int)blockIdx.x * share), c_end = min(a.H, c_begin + share);
  // every pass's steps, the routed experts' first
  const int routed = routed_passes * rs.steps, flat = routed + shared_passes * ss.steps;
  const int f0 = (int)((int64_t)flat * warp / kFewWarps);
  const int f1 = (int)((int64_t)flat * (warp + 1) / kFewWarps);
  const int d0 = f0 < routed ? f0 / rs.steps : routed_passes + (f0 - routed) / max(1, ss.steps);
  const int step0 = f0 < routed ? f0 % rs.steps : (f0 - routed) % max(1, ss.steps);
  const int dst = lane / 8 * 128;
  const uint32_t dst0 = dst + K::swizzle(lane / 8, lane % 8) * 16;
  const uint32_t dst1 = dst + 4 * 128 + K::swizzle(lane / 8 + 4, lane % 8) * 16;
  // units' first rows of h, and behind the last their number; then the rows' units and tokens
  const int* row0 = reinterpret_cast<const int*>(smem + a.p.row_at);
  const bool inside = a.p.hpitch > 0;
  bool waited = false;
  auto pass_at = [&](int d) {
    if constexpr (K::kPaired)
      return passes[d];
    else
      return FewPass{d, units[d].tokens};
  };

  for (int c0 = c_begin; c0 < c_end; c0 += 16 * kFewDownTiles) {
    const int channels = min(c_end - c0, 16 * kFewDownTiles);
    const int tiles = (channels + 15) / 16;
    // What is copied next: tile m of step next_step of pass next_d; the lane's piece of the
    // tile's row lane / 8, and the groups of the range's row lane / 2.
    int togo = f1 - f0, next_d = d0, next_step = step0, m_next = 0;
    int next_steps = 0, next_groups = 0, next_row = 0;
    const unsigned char *w = nullptr, *sp = nullptr, *zp = nullptr;
    int64_t four = 0;  // bytes of four rows
    auto enter = [&]() {
      const int e = units[pass_at(next_d).unit].expert;
      const FewMatrix& m = e < 0 ? a.shared[2] : a.m[2];
      next_steps = e < 0 ? ss.steps : rs.steps;
      next_groups = e < 0 ? ss.groups : rs.groups;
      next_row = e < 0 ? ss.row : rs.row;
      four = 4 * (int64_t)next_row;
      const int64_t first = (e < 0 ? 0 : (int64_t)e * a.H) + c0;
      w = m.w + (first + lane / 8) * next_row + next_step * 128 + (lane % 8) * 16;
      if constexpr (K::kFour) {
        const int64_t groups = (first + lane / 2) * next_groups;
        sp = m.s + groups * K::kScaleBytes;
        if constexpr (K::kZeros) zp = m.z + groups;
      }
    };
    if (togo) enter();
    auto issue = [&](uint32_t slot) {
      if (togo) {
        // rows past the range are not stored, whatever they hold
        int rows = channels - m_next * 16 - lane / 8;
        if (next_step * 128 + (lane % 8) * 16 >= next_row) rows = 0;
        copy_piece<K::kFour>(slot + dst0, w, rows > 0, a.x, policy);
        copy_piece<K::kFour>(slot + dst1, w + four, rows > 4, a.x, policy);
        copy_piece<K::kFour>(slot + dst0 + 8 * 128, w + 2 * four, rows > 8, a.x, policy);
        copy_piece<K::kFour>(slot + dst1 + 8 * 128, w + 3 * four, rows > 12, a.x, policy);
        if constexpr (K::kFour) {
          // (a row past the range takes the last one's)
          const int r = min(m_next * 16, channels - 1 - lane / 2) * next_groups;
          const unsigned char* z = nullptr;
          if constexpr (K::kZeros) z = zp + r;
          copy_groups<K>(a, next_groups, slot, next_step, sp + r * K::kScaleBytes, z);
        }
        w += 4 * four;
        if (++m_next == tiles) {
          w += 128 - tiles * 4 * four;
          m_next = 0;
          --togo;
          if (++next_step == next_steps) {
            next_step = 0;
            ++next_d;
            if (togo) enter();
          }
        }
      }
      cp_async_commit();
    };
    for (int i = 0; i < S - 1; ++i) issue(ring + i * sub);
    uint32_t use = ring, before = ring_last;
    if (!waited) {
      // every tile's h is stored (bounded: a tile belongs to a running team)
      if (tid == 0 && !wait_rows_done(&a.head->done, n.total))
        raise_status(a.status, kStTimeout, MOE_K_FEW_FFN);
      __syncthreads();
      waited = true;
      if (inside) {
        stage_h<K>(a, smem, units, row0[nunits], row0 + nunits + 1);
        __syncthreads();
      }
    }

    float acc[kFewDownTiles][4] = {}, total[kFewDownTiles][4] = {};
    float w0 = 0.f, w1 = 0.f, up = 1.f;
    bool in0 = false, in1 = false;  // tokens 2 tg and 2 tg + 1 are the pass's
    int from0 = 0, from1 = 0;       // their columns, where these are paired
    const float* hrow = nullptr;    // of the lane's column g
    uint32_t hat = 0;  // the row in shared memory
    FewGroups at{};  // of every tile: sixteen rows on, groups lie alike
    int d = d0, step = step0, steps = 0, kmax = 0;
    auto flush = [&]() {
#pragma unroll
      for (int m = 0; m < kFewDownTiles; ++m) {
        if constexpr (K::kPaired) {
          // columns c and c + 4 are the terms of the pass's token c: added, and brought to the
          // lane that has that token
          float both[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            both[i] = acc[m][i] + __shfl_xor_sync(0xffffffffu, acc[m][i], 2);
#pragma unroll
          for (int i = 0; i < 4; i += 2) {
            const float a0 = __shfl_sync(0xffffffffu, both[i], from0 / 2, 4);
            const float b0 = __shfl_sync(0xffffffffu, both[i + 1], from0 / 2, 4);
            const float a1 = __shfl_sync(0xffffffffu, both[i], from1 / 2, 4);
            const float b1 = __shfl_sync(0xffffffffu, both[i + 1], from1 / 2, 4);
            acc[m][i] = from0 & 1 ? b0 : a0;
            acc[m][i + 1] = from1 & 1 ? b1 : a1;
          }
        }
        // (other columns' sums are zeros, but NaN where a weight is not finite)
        if (in0) {
          total[m][0] = fmaf(w0, acc[m][0], total[m][0]);
          total[m][2] = fmaf(w0, acc[m][2], total[m][2]);
        }
        if (in1) {
          total[m][1] = fmaf(w1, acc[m][1], total[m][1]);
          total[m][3] = fmaf(w1, acc[m][3], total[m][3]);
        }
        acc[m][0] = acc[m][1] = acc[m][2] = acc[m][3] = 0.f;
      }
    };
    for (int f = f0; f < f1; ++f) {
      if (f == f0 || step == steps) {
        if (f > f0) {
          flush();
          step = 0;
          ++d;
        }
        const FewPass pass = pass_at(d);
        const int u = pass.unit, e = units[u].expert;
        const FewShape& sh = e < 0 ? ss : rs;
        steps = sh.steps;
        kmax = sh.K;
        const uint32_t tokens = pass.tokens;
        in0 = (tokens >> (2 * tg)) & 1u;
        in1 = (tokens >> (2 * tg + 1)) & 1u;
        int t = g;  // the token of the lane's column
        bool has = (tokens >> g) & 1u;
        if constexpr (K::kPaired) {  // the pass's token g % 4
          uint32_t left = tokens;
          for (int i = 0; i < g % kFewPairs; ++i) left &= left - 1u;
          has = left != 0u;
          t = has ? __ffs(left) - 1 : 0;
          from0 = __popc(tokens & ((1u << (2 * tg)) - 1u));
          from1 = from0 + in0;
        }
        hrow = has ? a.h + ((int64_t)u * a.T + t) * a.inter : nullptr;
        if (inside)
          hat = smem_u32(smem) + (row0[u] + __popc(units[u].tokens & ((1u << t) - 1u))) * a.p.hpitch +
                tg * 16 + (K::kPaired && g >= kFewPairs ? a.p.hrest : 0);
        w0 = __ldcg(&a.head->w[u][2 * tg]) * (K::kFour ? 16777216.f : 1.f);
        w1 = __ldcg(&a.head->w[u][2 * tg + 1]) * (K::kFour ? 16777216.f : 1.f);
        if constexpr (K::kScaled) {
          up = __uint_as_float(fp16_range_bits(__ldcg(&a.head->hmax[u][t])));
          w0 *= inverse_pow2(fp16_range_bits(__ldcg(&a.head->hmax[u][2 * tg])));
          w1 *= inverse_pow2(fp16_range_bits(__ldcg(&a.head->hmax[u][2 * tg + 1])));
        }
        at = groups_at<K>(a, sh, (e < 0 ? 0 : (int64_t)e * a.H) + c0 + g);
      }
      // the lane's h of this step, as MMA operands
      uint32_t b[K::kWords][4], rest[K::kRest ? K::kWords : 1][4];
      if (inside) {
#pragma unroll
        for (int i = 0; i < K::kWords; ++i) {
          uint4 v = make_uint4(0u, 0u, 0u, 0u), q = v;
          if (hrow) {
            v = lds128(hat + (step * (K::kStepK / 8) + K::piece(i, 0)) * 16);
            if constexpr (K::kRest)
              q = lds128(hat + a.p.hrest + (step * (K::kStepK / 8) + K::piece(i, 0)) * 16);
          }
          b[i][0] = v.x, b[i][1] = v.y, b[i][2] = v.z, b[i][3] = v.w;
          if constexpr (K::kRest) rest[i][0] = q.x, rest[i][1] = q.y, rest[i][2] = q.z, rest[i][3] = q.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < K::kWords; ++i) {
          const int k = step * K::kStepK + K::k_of(i, tg);
          float4 p = make_float4(0.f, 0.f, 0.f, 0.f), q = p;
          if (hrow && k < kmax) {
            p = __ldcg(reinterpret_cast<const float4*>(hrow + k));
            q = __ldcg(reinterpret_cast<const float4*>(hrow + k + 4));
          }
          h_operands<K>(p, q, up, b[i], rest[K::kRest ? i : 0]);
          if (K::kPaired && g >= kFewPairs) {
#pragma unroll
            for (int j = 0; j < 4; ++j) b[i][j] = rest[0][j];
          }
        }
      }
      float2 xs[K::kBlocks];
      if constexpr (K::kFour) {
#pragma unroll
        for (int blk = 0; blk < K::kBlocks; ++blk) {
          float d[4] = {};
          // sums: twos and thirty-twos (for what was divided by 16) of -2^-22, or -2^-25
          constexpr uint32_t kOne = K::kZeros ? 0x80018001u : 0x80088008u;   // -2^-24, -2^-21
          constexpr uint32_t kMany = K::kZeros ? 0x80108010u : 0x80808080u;  // 16 times that
#pragma unroll
          for (int i = 0; i < K::kPer; ++i) {
            mma16816<__half>(d, kOne, kOne, kMany, kMany, b[blk * K::kPer + i][0],
                             b[blk * K::kPer + i][1]);
            mma16816<__half>(d, kOne, kOne, kMany, kMany, b[blk * K::kPer + i][2],
                             b[blk * K::kPer + i][3]);
          }
          xs[blk] = make_float2(d[0], d[1]);
        }
      }
#pragma unroll
      for (int m = 0; m < kFewDownTiles; ++m) {
        if (m >= tiles) break;
        wait_stage(S);
        __syncwarp();
        issue(before);
        multiply<K, K::kRest>(use, b, rest, xs, a, at, step, acc[m]);
        before = use;
        use = use == ring_last ? ring : use + sub;
      }
      ++step;
      if constexpr (!K::kFour) {
        constexpr int kSteps = kFewChain / (4 * K::kWords);
        if ((f - f0) % kSteps == kSteps - 1) flush();
      }
    }
    flush();
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
      const int64_t col = c0 + c;
      const float zw = zero_w[t];
      if (zw != 0.f) {
        const uint16_t x = static_cast<const uint16_t*>(a.x)[t * a.ldx + col];
        v = fmaf(zw, a.fp16 ? __half2float(__ushort_as_half(x)) : bf16_to_f(x), v);
      }
      if (a.fp16)
        static_cast<__half*>(a.out)[t * a.ldo + col] = from_f<__half>(v);
      else
        static_cast<__nv_bfloat16*>(a.out)[t * a.ldo + col] = from_f<__nv_bfloat16>(v);
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
        K::order(v);
        q = make_uint4(pack2<__half>(v[0], v[1]), pack2<__half>(v[2], v[3]),
                       pack2<__half>(v[4], v[5]), pack2<__half>(v[6], v[7]));
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
      // what a block's sum starts from, in its unit of 2^-24: minus z x, z = 8 where the
      // zero points are not given
      sums[i] = fmaf(16.f, s16, s) * (K::kZeros ? -1.f : -8.f) * 0x1p-24f;
    }
    __syncthreads();
  }
}

template <typename K>
__global__ void __launch_bounds__(kFewThreads, 1) few_ffn_kernel(const __grid_constant__ FewArgs a) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ float x_inverse[kFewMaxT], zero_w[kFewMaxT];
  __shared__ int npasses[K::kPaired ? 2 : 1];  // of routed experts, of the shared one
  const int tid = threadIdx.x;
  // x is complete: the routing kernel let this one start only after its own wait for
  // everything before it.  What the routing kernel writes is read after the wait here.
  stage_x<K>(a, smem, x_inverse);
  pdl_wait();
  FewUnit* units = reinterpret_cast<FewUnit*>(smem + a.p.unit_at);
  const bool shared = a.Is > 0;
  FewTiles n;
  n.units = __ldcg(&a.head->units);
  n.routed = a.I / 8;
  n.shared = a.Is / 8;
  n.total = n.units * n.routed + n.shared;
  for (int i = tid; i < (n.units + shared) * (kFewUnitBytes / 4); i += kFewThreads)
    reinterpret_cast<uint32_t*>(units)[i] = __ldcg(reinterpret_cast<const uint32_t*>(a.head->unit) + i);
  if (tid < kFewMaxT) zero_w[tid] = __ldcg(&a.head->zero_w[tid]);
  __syncthreads();
  const int nunits = n.units + shared;
  if (a.p.hpitch > 0) {  // the rows of h (read after the next barrier)
    int* row0 = reinterpret_cast<int*>(smem + a.p.row_at);
    for (int u = tid; u <= nunits; u += kFewThreads) {
      int first = 0;
      for (int i = 0; i < u; ++i) first += __popc(units[i].tokens);
      row0[u] = first;
      if (u < nunits)
        for (int t = 0; t < kFewMaxT; ++t)
          if ((units[u].tokens >> t) & 1u) row0[nunits + 1 + first++] = u * kFewMaxT + t;
    }
  }
  gate_up<K>(a, smem, units, n, x_inverse);
  __syncthreads();
  pdl_trigger();
  FewPass* passes = reinterpret_cast<FewPass*>(smem + a.p.red_at);
  if constexpr (K::kPaired) {
    auto count = [&](int u) { return __popc(units[u].tokens) > kFewPairs ? 2 : 1; };
    for (int u = tid; u <= nunits; u += kFewThreads) {
      int at = 0;
      for (int i = 0; i < u; ++i) at += count(i);
      if (u == n.units) npasses[0] = at;
      if (u == n.units) npasses[1] = shared ? count(u) : 0;
      if (u < nunits) {
        uint32_t rest = units[u].tokens;
        for (int i = 0; i < kFewPairs; ++i) rest &= rest - 1u;
        passes[at] = {u, units[u].tokens ^ rest};
        if (rest) passes[at + 1] = {u, rest};
      }
    }
    __syncthreads();
  }
  const int routed = K::kPaired ? npasses[0] : n.units;
  down<K>(a, smem, units, n, passes, routed, K::kPaired ? npasses[1] : shared, nunits, zero_w);
}

// ------------------------------------------------------------------ launch --
template <int TT>
void launch_route(const Launch& L, const RouteArgs& r) {
  const int E = r.tk.E;
  const size_t need = route_scratch_inside(r.tk) ? (size_t)r.tk.T * E * 16 : 0;
  set_smem_attr_once(reinterpret_cast<const void*>(few_route_kernel<TT>), kRouteScratch,
                     kAttrFewRoute + (TT == 1 ? 0 : TT == 2 ? 1 : TT == 4 ? 2 : 3));
  launch_begin(L, MOE_K_FEW_ROUTE);
  launch_kernel(few_route_kernel<TT>, dim3(std::min(E, L.num_sms)), dim3(kRouteThreads), need,
                L.stream, r);
  launch_end(L, MOE_K_FEW_ROUTE);
}

template <typename K>
void launch_ffn(const Launch& L, const FewArgs& a, int slot) {
  set_smem_attr_once(reinterpret_cast<const void*>(few_ffn_kernel<K>), kFewSmem, kAttrFewFfn + slot);
  launch_begin(L, MOE_K_FEW_FFN);
  launch_kernel(few_ffn_kernel<K>, dim3(L.num_sms), dim3(kFewThreads), a.p.bytes, L.stream, a);
  launch_end(L, MOE_K_FEW_FFN);
}
template <int BLOCK, bool ZEROS, bool PAIRED>
void launch_four_as(const Launch& L, const FewArgs& a, int slot) {
  if (a.scale_dtype == MOE_DT_BF16)
    launch_ffn<Four<BLOCK, ZEROS, __nv_bfloat16, PAIRED>>(L, a, slot);
  else if (a.scale_dtype == MOE_DT_FP16)
    launch_ffn<Four<BLOCK, ZEROS, __half, PAIRED>>(L, a, slot + 1);
  else
    launch_ffn<Four<BLOCK, ZEROS, float, PAIRED>>(L, a, slot + 2);
}
template <int BLOCK>
void launch_four(const Launch& L, const FewArgs& a, bool zeros, int slot) {
  if (a.fp16) {
    if (zeros)
      launch_four_as<BLOCK, true, true>(L, a, slot);
    else
      launch_four_as<BLOCK, false, true>(L, a, slot + 3);
  } else if (zeros) {
    launch_four_as<BLOCK, true, false>(L, a, slot + 6);
  } else {
    launch_four_as<BLOCK, false, false>(L, a, slot + 9);
  }
}

// (without routed experts cfg.inter means nothing: it may be any number)
int few_inter(const moe_config& c) { return c.n_routed > 0 ? c.inter : 0; }

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
  l.total = l.h + up((size_t)units * T * std::max(few_inter(c), c.shared_inter) * 4);
  return l;
}

moe_status check_few(const moe_config* c, int T) {
  // the layer's own checks of the description; the batch's limits are this file's
  size_t bytes;
  const moe_status s = moe_workspace_size(c, T < 0 ? T : std::min(T, 1), &bytes);
  if (s != MOE_OK) return s;
  if (c->wdtype != MOE_W_BF16) return MOE_ERR_UNSUPPORTED;
  if (T > kFewMaxT || (int64_t)T * c->hidden > kFewMaxTH || few_inter(*c) > kFewMaxInter ||
      c->shared_inter > kFewMaxInter)
    return MOE_ERR_UNSUPPORTED;
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
  bool aligned_s = true, aligned_z = true, whole = true, zeros = false;
  if (four) {
    const int group = wt->group;
    if (group != 0 && group != 32 && group != 64 && group != 128) return MOE_ERR_INVALID_ARG;
    if (wt->scale_dtype < MOE_DT_BF16 || wt->scale_dtype > MOE_DT_FP32) return MOE_ERR_INVALID_ARG;
    const int es = wt->scale_dtype == MOE_DT_FP32 ? 4 : 2;
    for (int i = 0; i < 3; ++i) {
      const int k = i == 0 ? c.hidden : i == 1 ? few_inter(c) : c.shared_inter;
      if (k % 32 || (group > 0 && k % group)) return MOE_ERR_INVALID_ARG;
      const int groups = group > 0 ? k / group : 1;
      aligned_s = aligned_s && (k == 0 || groups * es % 4 == 0);
      aligned_z = aligned_z && (k == 0 || groups % 4 == 0);
      whole = whole && group > 0 && k % 256 == 0;
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
  if (out == x) return MOE_ERR_INVALID_ARG;

  FewArgs a{};
  const int units = std::min(c.n_routed, T * c.top_k) + (c.shared_inter > 0);
  const int es = wt->scale_dtype == MOE_DT_FP32 ? 4 : 2;
  a.p = few_plan(T, c.hidden, std::max(few_inter(c), c.shared_inter), units,
                 T * (std::min(c.n_routed, c.top_k) + (c.shared_inter > 0)), four, wt->group, es,
                 zeros, aligned_s, aligned_z, whole, !four || dtype == MOE_DT_FP16);
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
  a.I = few_inter(c);
  a.Is = c.shared_inter;
  a.inter = std::max(a.I, a.Is);  // a row of h: whole float4s
  a.fp16 = r.fp16;
  a.vec = r.vec;
  a.group = four ? wt->group : 0;
  a.scale_dtype = four ? wt->scale_dtype : MOE_DT_FP32;
  a.zstep = a.group ? a.p.step_k / a.group : 0;

  if (T == 1)
    launch_route<1>(L, r);
  else if (T == 2)
    launch_route<2>(L, r);
  else if (T <= 4)
    launch_route<4>(L, r);
  else
    launch_route<8>(L, r);
  if (!four && a.fp16)
    launch_ffn<Sixteen<__half>>(L, a, 0);
  else if (!four)
    launch_ffn<Sixteen<__nv_bfloat16>>(L, a, 1);
  else if (a.p.block == 32)
    launch_four<32>(L, a, zeros, 2);
  else if (a.p.block == 64)
    launch_four<64>(L, a, zeros, 14);
  else
    launch_four<128>(L, a, zeros, 26);
  return launch_status_take();
}
