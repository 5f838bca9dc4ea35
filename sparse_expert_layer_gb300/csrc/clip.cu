// Global norm of many tensors, and the tensors times min(1, max_norm / (norm + eps)).
//
// Two kernels: the sums of squares, then the products.  Each CTA has a contiguous part
// of the list of chunks of 32 KB; the first kernel goes through it forwards and the second
// backwards, so that what the first read last is still in L2 when the second starts there.
//
// Bound by memory where L2 can not hold the tensors: a product needs the norm, so they are read
// twice, 3 GB of bf16 in three tensors in 1370 us (two reads and a write: 1335 at 6.78 TB/s; 7.0 in
// the first kernel, 6.5 in the second).  Smaller ones wait for two launches with a sum of all slots
// between them: 48 fp32 tensors, 12.6 MB, 12.1 us (read and written once: 3.7); 37 tensors of all
// types, 40 MB, 22 (11.8).
//
// The squares of a thread's 64 elements of a chunk (fp32: 32) are added in fp32, its
// chunks and the threads as pairs of fp32, each CTA's sum in a slot of its own, and the slots
// in order: the same bits on every call on one device.
#include <math.h>

#include <algorithm>

#include "rows.cuh"

namespace moe {

namespace {

constexpr int kClipThreads = 256;
constexpr int kClipCtasPerSm = 4;
constexpr int kClipMaxCtas = 4096;   // slots of the workspace
constexpr int kClipUnroll = 8;       // 16-byte words of a thread in a chunk
constexpr int kClipChunk = kClipThreads * kClipUnroll;  // words
constexpr int kClipMost = 512;       // tensors of one launch
constexpr int kClipFew = 48;         // the same, for a short parameter block
constexpr int64_t kClipMaxElems = 1LL << 42;

struct ClipTensor {
  const unsigned char* in;   // down to a 16-byte boundary
  unsigned char* out;        // the byte that belongs to `in` (nullptr: not wanted)
  int64_t n;                 // bytes from `in` to the tensor's end
  int32_t skip;              // bytes from `in` to the tensor's first element
  int32_t dtype;
};

template <int N>
struct ClipList {
  ClipTensor t[N];
  int32_t first[N + 1];  // each tensor's first chunk
  int32_t count;
};

template <int N>
__device__ __forceinline__ int clip_find(const ClipList<N>& l, int chunk) {
  int lo = 0, hi = l.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (l.first[mid] <= chunk)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

template <typename T>
__device__ __forceinline__ void clip_unpack(const uint4& q, float (&x)[16 / sizeof(T)]) {
  if constexpr (sizeof(T) == 4) {
    memcpy(x, &q, 16);
  } else {
    const uint32_t p[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = unpack2<T>(p[j]);
      x[2 * j] = f.x;
      x[2 * j + 1] = f.y;
    }
  }
}
// The product with c, as it is stored.
template <typename T>
__device__ __forceinline__ uint4 clip_product(const uint4& q, float c) {
  constexpr int kPer = 16 / sizeof(T);
  float x[kPer];
  clip_unpack<T>(q, x);
  uint4 r;
  if constexpr (sizeof(T) == 4) {
    r = make_uint4(__float_as_uint(x[0] * c), __float_as_uint(x[1] * c), __float_as_uint(x[2] * c),
                   __float_as_uint(x[3] * c));
  } else {
    r = make_uint4(pack2<T>(x[0] * c, x[1] * c), pack2<T>(x[2] * c, x[3] * c),
                   pack2<T>(x[4] * c, x[5] * c), pack2<T>(x[6] * c, x[7] * c));
  }
  return r;
}

// The whole words of a chunk, as indexes into it, and an element in a word that a tensor begins
// or ends in, by the first threads.
struct ClipRange {
  int lo, hi;
  int64_t at;  // the element's byte
  bool edge;
  __device__ __forceinline__ ClipRange(const ClipTensor& t, int64_t word0) {
    const int64_t first = (t.skip + 15) / 16, last = t.n / 16;
    lo = (int)max((int64_t)0, first - word0);
    hi = (int)max((int64_t)0, min((int64_t)kClipChunk, last - word0));
    // threads 0 .. : elements of the first word, then of the last
    const int size = t.dtype == MOE_DT_FP32 ? 4 : 2, per = 16 / size;
    const bool front = threadIdx.x < per;
    const int64_t word = front ? 0 : last;
    at = word * 16 + (int)threadIdx.x % per * size;
    edge = threadIdx.x < 2 * per && at >= t.skip && at < t.n && word >= word0 &&
           word < word0 + kClipChunk && (front ? t.skip > 0 : last > 0 || t.skip == 0);
  }
};
__device__ __forceinline__ float clip_element(const unsigned char* p, int dtype) {
  if (dtype == MOE_DT_FP32) return *reinterpret_cast<const float*>(p);
  const uint16_t v = *reinterpret_cast<const uint16_t*>(p);
  return dtype == MOE_DT_BF16 ? bf16_to_f(v) : __half2float(__ushort_as_half(v));
}
__device__ __forceinline__ void clip_store(unsigned char* p, int dtype, float v) {
  if (dtype == MOE_DT_FP32)
    *reinterpret_cast<float*>(p) = v;
  else if (dtype == MOE_DT_BF16)
    *reinterpret_cast<__nv_bfloat16*>(p) = from_f<__nv_bfloat16>(v);
  else
    *reinterpret_cast<__half*>(p) = from_f<__half>(v);
}
// A thread's words of a chunk, all loads in flight (words outside are zeros).
__device__ __forceinline__ void clip_load(const ClipTensor& t, int64_t word0, const ClipRange& r,
                                          uint4 (&v)[kClipUnroll]) {
  const uint4* p = reinterpret_cast<const uint4*>(t.in) + word0;
#pragma unroll
  for (int i = 0; i < kClipUnroll; ++i) {
    const int w = threadIdx.x + i * kClipThreads;
    v[i] = w >= r.lo && w < r.hi ? p[w] : make_uint4(0u, 0u, 0u, 0u);
  }
}

template <typename T>
__device__ __forceinline__ float clip_squares(const uint4 (&v)[kClipUnroll]) {
  constexpr int kPer = 16 / sizeof(T);
  float s[4] = {};
#pragma unroll
  for (int i = 0; i < kClipUnroll; ++i) {
    float x[kPer];
    clip_unpack<T>(v[i], x);
#pragma unroll
    for (int j = 0; j < kPer; ++j) s[j % 4] = fmaf(x[j], x[j], s[j % 4]);
  }
  return (s[0] + s[1]) + (s[2] + s[3]);
}
template <typename T>
__device__ __forceinline__ void clip_products(uint4* o, const ClipRange& r,
                                              const uint4 (&v)[kClipUnroll], float c) {
#pragma unroll
  for (int i = 0; i < kClipUnroll; ++i) {
    const int w = threadIdx.x + i * kClipThreads;
    if (w >= r.lo && w < r.hi) o[w] = clip_product<T>(v[i], c);
  }
}

__device__ __forceinline__ float clip_square(const ClipTensor& t, const ClipRange& r,
                                             const uint4 (&v)[kClipUnroll]) {
  float x = 0.f;
  if (r.edge) x = clip_element(t.in + r.at, t.dtype);
  const float s = t.dtype == MOE_DT_BF16   ? clip_squares<__nv_bfloat16>(v)
                  : t.dtype == MOE_DT_FP16 ? clip_squares<__half>(v)
                                           : clip_squares<float>(v);
  return fmaf(x, x, s);
}

__device__ __forceinline__ void clip_scale(const ClipTensor& t, int64_t word0, const ClipRange& r,
                                           const uint4 (&v)[kClipUnroll], float c) {
  if ((reinterpret_cast<uintptr_t>(t.out) & 15u) == 0) {
    uint4* o = reinterpret_cast<uint4*>(t.out) + word0;
    if (t.dtype == MOE_DT_BF16)
      clip_products<__nv_bfloat16>(o, r, v, c);
    else if (t.dtype == MOE_DT_FP16)
      clip_products<__half>(o, r, v, c);
    else
      clip_products<float>(o, r, v, c);
  } else {  // out begins at another byte of a word than in
    const int size = t.dtype == MOE_DT_FP32 ? 4 : 2;
    for (int64_t b = (word0 + r.lo) * 16 + threadIdx.x * size; b < (word0 + r.hi) * 16;
         b += kClipThreads * size)
      clip_store(t.out + b, t.dtype, clip_element(t.in + b, t.dtype) * c);
  }
  if (r.edge) clip_store(t.out + r.at, t.dtype, clip_element(t.in + r.at, t.dtype) * c);
}

// A CTA's chunks, a contiguous part of the list, forwards or backwards.  The tensor that they
// belong to is looked up once, kept in registers and then followed: indexed reads of the
// parameters are slow (read for every chunk they took longer than 20 MB of data).
template <int N, bool BACK>
struct ClipWalk {
  const ClipList<N>& l;
  ClipTensor t;
  int chunk, left, i, begin, end;  // begin, end: the tensor's chunks
  __device__ __forceinline__ ClipWalk(const ClipList<N>& list) : l(list) {
    const int64_t chunks = l.first[l.count];
    const int c0 = (int)(chunks * blockIdx.x / gridDim.x);
    const int c1 = (int)(chunks * (blockIdx.x + 1) / gridDim.x);
    left = c1 - c0;
    chunk = BACK ? c1 - 1 : c0;
    i = left > 0 ? clip_find(l, chunk) : 0;
    enter();
  }
  __device__ __forceinline__ void enter() {
    t = l.t[i];
    begin = l.first[i];
    end = l.first[i + 1];
  }
  __device__ __forceinline__ int64_t word() const { return (int64_t)(chunk - begin) * kClipChunk; }
  __device__ __forceinline__ void next() {
    --left;
    chunk += BACK ? -1 : 1;
    if (left > 0 && (BACK ? chunk < begin : chunk >= end)) {
      i += BACK ? -1 : 1;
      enter();
    }
  }
};

// A sum as hi + lo, lo the rounding errors of hi's additions (Knuth's exact addition).  fp64
// would do it shorter, but its rate here is so low that with it 12.6 MB took 19.7 us instead of 12.1.  hi is inf or NaN where the sum is; lo means nothing then.
struct ClipSum {
  float hi, lo;
};
__device__ __forceinline__ ClipSum clip_add(const ClipSum& a, const ClipSum& b) {
  const float s = a.hi + b.hi, t = s - a.hi;
  return {s, ((a.hi - (s - t)) + (b.hi - t)) + (a.lo + b.lo)};
}
// The root of a sum, as a pair too: one Newton step from the rounded root.
__device__ __forceinline__ ClipSum clip_root(const ClipSum& a) {
  const float r = sqrtf(a.hi), e = (fmaf(-r, r, a.hi) + a.lo) / (2.f * r);
  return {r, fabsf(e) <= r * 0x1p-20f ? e : 0.f};  // none of 0, inf and NaN
}
// min(1, max_norm / (norm + eps)), rounded once: every element's product has its error, which
// a rounded sum, quotient and root would make three times that.  NaN stays one.
__device__ __forceinline__ float clip_factor(const ClipSum& norm, float max_norm, float eps) {
  const ClipSum d = clip_add(norm, {eps, 0.f});
  const float q = max_norm / d.hi;
  const float e = (fmaf(-q, d.hi, max_norm) - q * d.lo) / d.hi;
  const float c = fabsf(e) <= q * 0x1p-20f ? q + e : q;
  return c >= 1.f ? 1.f : c;
}
// The block's sum of v, in every thread; added in a fixed order.
__device__ __forceinline__ ClipSum clip_block_sum(ClipSum v) {
  __shared__ ClipSum part[kClipThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    v = clip_add(v, {__shfl_xor_sync(0xffffffffu, v.hi, o), __shfl_xor_sync(0xffffffffu, v.lo, o)});
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
  __syncthreads();
  ClipSum s = part[0];
#pragma unroll
  for (int i = 1; i < kClipThreads / 32; ++i) s = clip_add(s, part[i]);
  return s;
}

// more: a list after the first one, added to what the slots hold.
template <int N>
__global__ void __launch_bounds__(kClipThreads, kClipCtasPerSm)
    clip_norm_kernel(const __grid_constant__ ClipList<N> l, ClipSum* slots, int more) {
  pdl_enter();
  ClipSum sum{0.f, 0.f};
  for (ClipWalk<N, false> walk(l); walk.left > 0; walk.next()) {
    const ClipRange r(walk.t, walk.word());
    uint4 v[kClipUnroll];
    clip_load(walk.t, walk.word(), r, v);
    sum = clip_add(sum, {clip_square(walk.t, r, v), 0.f});
  }
  sum = clip_block_sum(sum);
  if (threadIdx.x == 0) slots[blockIdx.x] = more ? clip_add(slots[blockIdx.x], sum) : sum;
}

template <int N>
__global__ void __launch_bounds__(kClipThreads, kClipCtasPerSm)
    clip_scale_kernel(const __grid_constant__ ClipList<N> l, const ClipSum* slots, int nslots,
                      float max_norm, float eps, float* norm_out) {
  pdl_enter();
  ClipSum sum{0.f, 0.f};
  for (int i = threadIdx.x; i < nslots; i += kClipThreads) sum = clip_add(sum, slots[i]);
  const ClipSum norm = clip_root(clip_block_sum(sum));
  if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = norm.hi + norm.lo;
  const float c = clip_factor(norm, max_norm, eps);
  for (ClipWalk<N, true> walk(l); walk.left > 0; walk.next()) {
    if (!walk.t.out || (c == 1.f && walk.t.out == walk.t.in)) continue;
    const ClipRange r(walk.t, walk.word());
    uint4 v[kClipUnroll];
    clip_load(walk.t, walk.word(), r, v);
    clip_scale(walk.t, walk.word(), r, v, c);
  }
}

int clip_size(int dtype) { return dtype == MOE_DT_FP32 ? 4 : 2; }

// Tensors [i, i + count) of the call; false: more chunks than an int counts.
template <int N>
bool clip_list(const moe_tensor* ts, int count, ClipList<N>* l) {
  int64_t chunks = 0;
  l->count = 0;
  for (int i = 0; i < count; ++i) {
    const moe_tensor& s = ts[i];
    if (s.n == 0) continue;
    ClipTensor& t = l->t[l->count];
    const uintptr_t at = reinterpret_cast<uintptr_t>(s.in);
    t.skip = (int32_t)(at & 15u);
    t.in = reinterpret_cast<const unsigned char*>(at - t.skip);
    t.out = s.out ? static_cast<unsigned char*>(s.out) - t.skip : nullptr;
    t.n = t.skip + s.n * clip_size(s.dtype);
    t.dtype = s.dtype;
    l->first[l->count++] = (int32_t)chunks;
    chunks += (t.n + kClipChunk * 16LL - 1) / (kClipChunk * 16LL);
    if (chunks > INT32_MAX - kClipMaxCtas) return false;
  }
  l->first[l->count] = (int32_t)chunks;
  return true;
}

template <int N>
moe_status clip_run(const Launch& L, int n, const moe_tensor* ts, float max_norm, float eps,
                    float* norm, ClipSum* slots) {
  const int most = std::min(kClipMaxCtas, kClipCtasPerSm * L.num_sms);
  ClipList<N> l;
  // every list has the slots of all CTAs, so that later lists add to what is there
  int used = 0;
  for (int i = 0; i < n; i += N) {
    if (!clip_list<N>(ts + i, std::min(N, n - i), &l)) return MOE_ERR_UNSUPPORTED;
    used = std::max(used, std::min(most, l.first[l.count]));
  }
  used = std::max(used, 1);
  for (int pass = 0; pass < 2; ++pass) {
    bool scaled = pass == 0 || norm != nullptr;
    for (int i = 0; i < n && !scaled; ++i) scaled = ts[i].out != nullptr && ts[i].n > 0;
    if (!scaled) break;
    for (int i = 0; i < std::max(n, 1); i += N) {
      // the second pass goes backwards
      const int last = (std::max(n, 1) - 1) / N * N, at = pass ? last - i : i;
      clip_list<N>(ts + at, std::min(N, n - at), &l);
      launch_begin(L, pass ? MOE_K_CLIP : MOE_K_GRAD_NORM);
      if (pass == 0)
        launch_kernel(clip_norm_kernel<N>, dim3(used), dim3(kClipThreads), 0, L.stream, l, slots,
                      at > 0 ? 1 : 0);
      else
        launch_kernel(clip_scale_kernel<N>, dim3(used), dim3(kClipThreads), 0, L.stream, l,
                      static_cast<const ClipSum*>(slots), used, max_norm, eps,
                      i == 0 ? norm : nullptr);
      launch_end(L, pass ? MOE_K_CLIP : MOE_K_GRAD_NORM);
    }
  }
  return launch_status_take();
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_clip_workspace_size(size_t* bytes) {
  if (!bytes) return MOE_ERR_INVALID_ARG;
  *bytes = kClipMaxCtas * sizeof(ClipSum);
  return MOE_OK;
}

extern "C" moe_status moe_clip_grad_norm(int32_t n, const moe_tensor* tensors, float max_norm,
                                         float eps, float* norm, void* ws, size_t ws_bytes,
                                         moe_stream_t stream) {
  if (n < 0 || (n > 0 && !tensors) || !isfinite(max_norm) || max_norm < 0.f || !isfinite(eps) ||
      eps < 0.f)
    return MOE_ERR_INVALID_ARG;
  bool outputs = norm != nullptr;
  for (int i = 0; i < n; ++i) {
    const moe_tensor& t = tensors[i];
    if (t.n < 0 || t.dtype < MOE_DT_BF16 || t.dtype > MOE_DT_FP32) return MOE_ERR_INVALID_ARG;
    if (t.n > kClipMaxElems) return MOE_ERR_UNSUPPORTED;
    if (t.n > 0 && !t.in) return MOE_ERR_INVALID_ARG;
    const uintptr_t mask = clip_size(t.dtype) - 1;
    if ((reinterpret_cast<uintptr_t>(t.in) & mask) || (reinterpret_cast<uintptr_t>(t.out) & mask))
      return MOE_ERR_ALIGNMENT;
    outputs = outputs || t.out;
  }
  if (!outputs) return MOE_ERR_INVALID_ARG;
  if (!ws) return MOE_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(ws) & 255u) || (reinterpret_cast<uintptr_t>(norm) & 3u))
    return MOE_ERR_ALIGNMENT;
  if (ws_bytes < kClipMaxCtas * sizeof(ClipSum)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  Launch L;
  const moe_status s = open_launch(stream, &L);
  if (s != MOE_OK) return s;
  ClipSum* slots = static_cast<ClipSum*>(ws);
  return n <= kClipFew ? clip_run<kClipFew>(L, n, tensors, max_norm, eps, norm, slots)
                       : clip_run<kClipMost>(L, n, tensors, max_norm, eps, norm, slots);
}
