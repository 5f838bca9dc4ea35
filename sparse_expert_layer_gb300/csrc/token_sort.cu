// Tokens sorted by expert and back, with the gradients of both.
//
// Pick r = t * k + j of token t goes to the bucket of its expert, or to a last
// bucket of dropped picks when its id is outside [0, E) (a masked slot, or an
// expert held elsewhere).  Buckets follow each other, and inside a bucket the
// picks keep their order, so the sorted positions are a permutation of the T * k
// picks with the kept ones first:
//   position(r) = #{r' : key' < key} + #{r' < r : key' == key}.
//
// Rows move token by token: a token's row is read once and written to its k
// positions, and on the way back its k rows are read and added in slot order in
// fp32, so no result depends on the order in which CTAs run.
//
// All of it is bound by memory once the batch is large: sorting 8192 tokens x 8
// picks of 7168 bf16 channels moves 1.06 GB in 171 us (6.2 TB/s, 91% of the copy
// rate), the gradients of 4096 x 8 x 5120 1.09 GB in 173 us (93%).  Small batches
// are launches and latency: 64 tokens x 12 picks 5.3 us in one launch.
#include <algorithm>
#include <climits>

#include "rows.cuh"

namespace moe {

namespace {

constexpr int kSortMaxExperts = 4096;
constexpr int kSortMaxTopK = 32;
constexpr int kSortThreads = 256;
constexpr int kSortBlockPicks = 256;  // most picks one CTA of the counting passes takes
// Small batches: every CTA finds its token's positions by itself, reading all
// ids; T CTAs compare R picks each, so the limit is on T * R too.  One launch
// against four: 512 tokens x 8 picks 7.5 against 9.7 us, 1400 x 1 7.9 against 9.7,
// but 1024 x 4 11.3 against 10.1 (rows of 1024 bf16 channels).
constexpr int kSortDirectPicks = 4096;
constexpr int64_t kSortDirectWork = 1 << 21;
bool sort_direct(int64_t T, int64_t k) {
  return T * k <= kSortDirectPicks && T * T * k <= kSortDirectWork;
}

__device__ __forceinline__ int pick_key(int32_t id, int E) {
  return (unsigned)id < (unsigned)E ? id : E;
}

struct RowsArgs {
  const unsigned char* x;
  unsigned char* out;
  const float* x_scale;
  float* out_scale;
  int64_t ldx, ldo;  // bytes
  int units;         // copy units of a row
  int zero_dropped;
};

// Copies units [first, last) of token t's row to the k sorted rows pos[j];
// positions from `kept` on belong to dropped picks.
template <typename U>
__device__ __forceinline__ void copy_row(const RowsArgs& a, int t, int k, const int* pos, int kept,
                                         int first, int last, int tid, int stride) {
  const U* src = reinterpret_cast<const U*>(a.x + (int64_t)t * a.ldx);
  for (int i = first + tid; i < last; i += stride) {
    const U v = src[i];
    for (int j = 0; j < k; ++j) {
      const int p = pos[j];
      U* dst = reinterpret_cast<U*>(a.out + (int64_t)p * a.ldo) + i;
      if (p < kept)
        *dst = v;
      else if (a.zero_dropped)
        *dst = U{};
    }
  }
  if (a.out_scale && first == 0)
    for (int j = tid; j < k; j += stride) {
      if (pos[j] < kept)
        a.out_scale[pos[j]] = a.x_scale[t];
      else if (a.zero_dropped)
        a.out_scale[pos[j]] = 0.f;
    }
}

struct PlanArgs {
  const int32_t* ids;
  int32_t* counts;
  int32_t* offsets;
  int32_t* s2e;
  int32_t* e2s;
  int32_t* table;  // counting passes: [E + 1][nblk]
  int T, k, E, nblk, tokens;  // tokens of a counting block
};

// ------------------------------------------------------------ one launch --
// Key and index of a pick as one number: picks compare as their positions do.
__device__ __forceinline__ uint32_t pick_order(int32_t id, int i, int E, int R) {
  return (uint32_t)pick_key(id, E) * (uint32_t)R + (uint32_t)i;
}
constexpr int kDirectBatch = 8;  // picks counted in one reading of the ids

// The first T * chunks CTAs each take a chunk of one token's row; the rest find
// the experts' counts and offsets, a warp an expert.  Every CTA reads all R ids.
template <typename U>
__global__ void __launch_bounds__(kSortThreads)
    sort_direct_kernel(PlanArgs p, RowsArgs a, int chunks, int chunk_units) {
  pdl_enter();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  constexpr int kWarps = kSortThreads / 32;
  const int R = p.T * p.k;
  const int row_blocks = p.T * chunks;
  if ((int)blockIdx.x >= row_blocks) {
    const int e = ((int)blockIdx.x - row_blocks) * kWarps + warp;
    if (e > p.E) return;
    int below = 0, same = 0;
    auto take = [&](int32_t id) {
      const int key = pick_key(id, p.E);
      below += key < e;
      same += key == e;
    };
    const int quads = R / 4;
#pragma unroll 4
    for (int i = lane; i < quads; i += 32) {
      const int4 v = reinterpret_cast<const int4*>(p.ids)[i];
      take(v.x);
      take(v.y);
      take(v.z);
      take(v.w);
    }
    if (4 * quads + lane < R) take(p.ids[4 * quads + lane]);
    below = __reduce_add_sync(0xffffffffu, below);
    same = __reduce_add_sync(0xffffffffu, same);
    if (lane == 0) {
      p.offsets[e] = below;
      if (e < p.E) p.counts[e] = same;
    }
    return;
  }
  __shared__ int pos[kSortMaxTopK + 1];  // the last: the number of kept picks
  __shared__ int part[kWarps][kSortMaxTopK + 1];
  const int t = blockIdx.x / chunks, c = blockIdx.x % chunks;
  for (int j0 = 0; j0 < p.k; j0 += kDirectBatch) {
    uint32_t limit[kDirectBatch];
    int n[kDirectBatch] = {}, kept = 0;
#pragma unroll
    for (int b = 0; b < kDirectBatch; ++b) {
      const int r = t * p.k + j0 + b;
      limit[b] = j0 + b < p.k ? pick_order(p.ids[r], r, p.E, R) : 0u;
    }
    const uint32_t dropped = (uint32_t)p.E * (uint32_t)R;
#pragma unroll 4
    for (int i = threadIdx.x; i < R; i += kSortThreads) {
      const uint32_t order = pick_order(p.ids[i], i, p.E, R);
      kept += order < dropped;
#pragma unroll
      for (int b = 0; b < kDirectBatch; ++b) n[b] += order < limit[b];
    }
#pragma unroll
    for (int b = 0; b < kDirectBatch; ++b) {
      const int all = __reduce_add_sync(0xffffffffu, n[b]);
      if (lane == b && j0 + b < p.k) part[warp][j0 + b] = all;
    }
    if (j0 == 0) {
      kept = __reduce_add_sync(0xffffffffu, kept);
      if (lane == 0) part[warp][p.k] = kept;
    }
  }
  __syncthreads();
  if (threadIdx.x <= p.k) {
    int sum = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += part[w][threadIdx.x];
    pos[threadIdx.x] = sum;
  }
  __syncthreads();
  if (c == 0 && threadIdx.x < p.k) {
    const int r = t * p.k + threadIdx.x, at = pos[threadIdx.x];
    p.e2s[r] = at;
    p.s2e[at] = r;
  }
  if (!a.out) return;
  const int first = c * chunk_units;
  copy_row<U>(a, t, p.k, pos, pos[p.k], first, min(a.units, first + chunk_units), threadIdx.x,
              kSortThreads);
}

// ------------------------------------------------------- counting passes --
__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(PlanArgs p) {
  pdl_enter();
  extern __shared__ int32_t hist[];  // [E + 1]
  for (int e = threadIdx.x; e <= p.E; e += kSortThreads) hist[e] = 0;
  __syncthreads();
  const int b = blockIdx.x;
  const int r0 = b * p.tokens * p.k, r1 = min(p.T, (b + 1) * p.tokens) * p.k;
  for (int r = r0 + threadIdx.x; r < r1; r += kSortThreads)
    atomicAdd(&hist[pick_key(p.ids[r], p.E)], 1);
  __syncthreads();
  for (int e = threadIdx.x; e <= p.E; e += kSortThreads)
    p.table[(size_t)e * p.nblk + b] = hist[e];
}

// One warp an expert: its blocks' counts -> how many of its picks lie in
// earlier blocks.
__global__ void __launch_bounds__(kSortThreads) sort_scan_kernel(PlanArgs p) {
  pdl_enter();
  const int lane = threadIdx.x % 32;
  const int e = blockIdx.x * (kSortThreads / 32) + threadIdx.x / 32;
  if (e > p.E) return;
  int32_t* row = p.table + (size_t)e * p.nblk;
  int carry = 0;
  for (int b0 = 0; b0 < p.nblk; b0 += 32) {
    const int b = b0 + lane;
    const int v = b < p.nblk ? row[b] : 0;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int n = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += n;
    }
    if (b < p.nblk) row[b] = carry + incl - v;
    carry += __shfl_sync(0xffffffffu, incl, 31);
  }
  if (lane == 0 && e < p.E) p.counts[e] = carry;
}

// Every CTA scans the counts for itself, then places its block's picks.
__global__ void __launch_bounds__(kSortThreads) sort_place_kernel(PlanArgs p) {
  pdl_enter();
  extern __shared__ int32_t off[];  // [E + 1]
  __shared__ __align__(16) int32_t keys[kSortBlockPicks];
  __shared__ int32_t wsum[kSortThreads / 32];
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  int carry = 0;
  for (int base = 0; base <= p.E; base += kSortThreads) {
    const int e = base + tid;
    const int v = e < p.E ? p.counts[e] : 0;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int n = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += n;
    }
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    int before = carry, all = 0;
#pragma unroll
    for (int w = 0; w < kSortThreads / 32; ++w) {
      if (w < warp) before += wsum[w];
      all += wsum[w];
    }
    if (e <= p.E) {
      off[e] = before + incl - v;
      if (blockIdx.x == 0) p.offsets[e] = before + incl - v;
    }
    carry += all;
    __syncthreads();
  }
  const int b = blockIdx.x;
  const int r0 = b * p.tokens * p.k, n = min(p.T, (b + 1) * p.tokens) * p.k - r0;
  if (tid < n) keys[tid] = pick_key(p.ids[r0 + tid], p.E);
  __syncthreads();
  if (tid < n) {
    const int key = keys[tid];
    int at = off[key] + p.table[(size_t)key * p.nblk + b];
    int i = 0;
    for (; i + 4 <= tid; i += 4) {
      const int4 v = *reinterpret_cast<const int4*>(keys + i);
      at += (v.x == key) + (v.y == key) + (v.z == key) + (v.w == key);
    }
    for (; i < tid; ++i) at += keys[i] == key;
    p.s2e[at] = r0 + tid;
    p.e2s[r0 + tid] = at;
  }
}

template <typename U>
__global__ void __launch_bounds__(kSortThreads)
    sort_rows_kernel(RowsArgs a, const int32_t* e2s, const int32_t* offsets, int k, int E,
                     int chunks, int chunk_units) {
  pdl_enter();
  __shared__ int pos[kSortMaxTopK];
  const int t = blockIdx.x / chunks, c = blockIdx.x % chunks;
  if (threadIdx.x < k) pos[threadIdx.x] = e2s[(size_t)t * k + threadIdx.x];
  const int kept = offsets[E];
  __syncthreads();
  const int first = c * chunk_units;
  copy_row<U>(a, t, k, pos, kept, first, min(a.units, first + chunk_units), threadIdx.x,
              kSortThreads);
}

// ------------------------------------------------------------- way back --
struct BackArgs {
  const void* rows;   // [R, H] sorted rows
  const int32_t* offsets;
  const int32_t* e2s;
  const float* w;     // [T, k], nullptr: ones
  void* out;          // [T, H]
  int64_t ldo;        // elements
  int T, k, E, H, nslots;
};

constexpr int kBackBatch = 4;  // picks whose rows are loaded before any is added

// out[t] = sum over the token's kept picks, in slot order, of w * row.
template <typename TI, typename TO, bool VEC>
__global__ void __launch_bounds__(128) unsort_kernel(BackArgs a, int chunks) {
  pdl_enter();
  __shared__ int pos[kSortMaxTopK];
  __shared__ float wts[kSortMaxTopK];
  const int t = blockIdx.x / chunks, c = blockIdx.x % chunks;
  if (threadIdx.x < a.k) {
    const size_t r = (size_t)t * a.k + threadIdx.x;
    const int p = a.e2s[r];
    // a position outside the kept rows (a dropped pick) is skipped
    pos[threadIdx.x] = p >= 0 && p < min(a.offsets[a.E], a.T * a.k) ? p : -1;
    wts[threadIdx.x] = a.w ? a.w[r] : 1.f;
  }
  __syncthreads();
  const int s = c * blockDim.x + threadIdx.x;
  if (!slot_inside<!VEC>(s, a.nslots)) return;
  float acc[kSlot] = {};
  for (int j0 = 0; j0 < a.k; j0 += kBackBatch) {
    Raw8<TI> raw[kBackBatch];
#pragma unroll
    for (int b = 0; b < kBackBatch; ++b) {
      const int p = j0 + b < a.k ? pos[j0 + b] : -1;
      if (p >= 0)
        raw[b] = load_raw8<TI, VEC>(static_cast<const TI*>(a.rows) + (int64_t)p * a.H, s, a.H);
    }
#pragma unroll
    for (int b = 0; b < kBackBatch; ++b) {
      if (j0 + b >= a.k || pos[j0 + b] < 0) continue;
      float f[kSlot];
      unpack8<TI>(raw[b], f);
      const float wj = wts[j0 + b];
#pragma unroll
      for (int i = 0; i < kSlot; ++i) acc[i] = fmaf(wj, f[i], acc[i]);
    }
  }
  store8<TO, VEC>(static_cast<TO*>(a.out) + (int64_t)t * a.ldo, s, a.H, acc);
}

struct GradArgs {
  const void* dout;   // [T, H]
  const void* rows;   // [R, H] sorted rows of the forward pass
  const int32_t* offsets;
  const int32_t* e2s;
  const float* w;
  void* drows;        // [R, H], nullptr: not wanted
  float* dw;          // [T, k]
  int64_t ldd;        // elements
  int T, k, E, H, nslots;
  int picks;          // picks one CTA takes
  int zero_dropped;
};

constexpr int kGradThreads = 256;

// drows[p] = w * dout[t], dw = <dout[t], rows[p]>: a CTA takes `picks` picks of
// one token; a slot of dout is loaded once for all of them.  A thread's channels
// are neighbours in rows of any alignment: dw has the same bits whatever the row
// strides.  Rows of odd lengths pay for that with accesses of one channel, eight
// channels apart in a warp: 2048 x 8 of 5121 bf16 channels take 161 us (33% of the
// copy rate), of 5120 63 us.  ROWS false: drows is not wanted (4096 x 8 of 5120 bf16 channels take
// 68 us instead of 119).  A test at run time instead cost rows of odd lengths 7%.
template <typename TI, typename TO, bool VEC, bool ROWS>
__global__ void __launch_bounds__(kGradThreads) unsort_grad_kernel(GradArgs a, int parts) {
  pdl_enter();
  constexpr int kWarps = kGradThreads / 32;
  __shared__ int pos[kSortMaxTopK];
  __shared__ float wts[kSortMaxTopK];
  __shared__ float dots[kWarps][kSortMaxTopK];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int t = blockIdx.x / parts, j_first = (blockIdx.x % parts) * a.picks;
  const int nj = min(a.picks, a.k - j_first);
  const int R = a.T * a.k, kept = min(a.offsets[a.E], R);
  if (threadIdx.x < nj) {
    const size_t r = (size_t)t * a.k + j_first + threadIdx.x;
    pos[threadIdx.x] = a.e2s[r];
    wts[threadIdx.x] = a.w[r];
  }
  for (int i = threadIdx.x; i < kWarps * kSortMaxTopK; i += kGradThreads)
    dots[i / kSortMaxTopK][i % kSortMaxTopK] = 0.f;
  __syncthreads();
  for (int s0 = 0; s0 < a.nslots; s0 += kGradThreads) {
    const int s = s0 + threadIdx.x;
    const bool in = s < a.nslots;
    float d[kSlot] = {};
    if (in) load8<TO, VEC, false>(static_cast<const TO*>(a.dout) + (int64_t)t * a.ldd, s, a.H, d);
    for (int j0 = 0; j0 < nj; j0 += kBackBatch) {
      Raw8<TI> raw[kBackBatch];
#pragma unroll
      for (int b = 0; b < kBackBatch; ++b) {
        const int p = j0 + b < nj ? pos[j0 + b] : -1;
        if (in && p >= 0 && p < kept)
          raw[b] = load_raw8<TI, VEC, false>(static_cast<const TI*>(a.rows) + (int64_t)p * a.H, s, a.H);
      }
#pragma unroll
      for (int b = 0; b < kBackBatch; ++b) {
        if (j0 + b >= nj) continue;
        const int p = pos[j0 + b];
        float dot = 0.f;
        if (in && p >= 0 && p < R) {
          const bool use = p < kept;
          float f[kSlot];
          if (use) {
            unpack8<TI>(raw[b], f);
#pragma unroll
            for (int i = 0; i < kSlot; ++i) dot = fmaf(d[i], f[i], dot);
          }
          if constexpr (ROWS) {
            float g[kSlot];
#pragma unroll
            for (int i = 0; i < kSlot; ++i) g[i] = use ? wts[j0 + b] * d[i] : 0.f;
            if (use || a.zero_dropped)
              store8<TI, VEC, false>(static_cast<TI*>(a.drows) + (int64_t)p * a.H, s, a.H, g);
          }
        }
        dot = warp_sum(dot);
        if (lane == 0) dots[warp][j0 + b] += dot;
      }
    }
  }
  __syncthreads();
  if (threadIdx.x < nj) {
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += dots[w][threadIdx.x];
    a.dw[(size_t)t * a.k + j_first + threadIdx.x] = sum;
  }
}

// --------------------------------------------------------------- host side --
int dtype_bytes(int32_t dt) {
  switch (dt) {
    case MOE_DT_BF16:
    case MOE_DT_FP16: return 2;
    case MOE_DT_FP32: return 4;
    case MOE_DT_INT8:
    case MOE_DT_E4M3: return 1;
  }
  return 0;
}

moe_status check_sort(int32_t T, int32_t k, int32_t E) {
  if (T < 0 || k < 1 || E < 1) return MOE_ERR_INVALID_ARG;
  if (k > kSortMaxTopK || E > kSortMaxExperts || (int64_t)T * k > (1LL << 30))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

int block_tokens(int k) { return kSortBlockPicks / k; }
int block_count(int T, int k) { return (T + block_tokens(k) - 1) / block_tokens(k); }

// Row chunks so that about two CTAs run on every SM, of at least one unit a thread.
int row_chunks(int T, int units, int threads, int num_sms) {
  const int most = (units + threads - 1) / threads;
  const int want = (2 * num_sms + T - 1) / T;
  return std::max(1, std::min(most, want));
}

template <typename U>
void launch_sort(const Launch& L, PlanArgs p, RowsArgs a) {
  const int chunks = a.out ? row_chunks(p.T, a.units, kSortThreads, L.num_sms) : 1;
  const int chunk_units = a.out ? (a.units + chunks - 1) / chunks : 0;
  if (sort_direct(p.T, p.k)) {
    const int grid = p.T * chunks + (p.E + 1 + kSortThreads / 32 - 1) / (kSortThreads / 32);
    launch_begin(L, MOE_K_SORT_ROWS);
    launch_kernel(sort_direct_kernel<U>, grid, kSortThreads, 0, L.stream, p, a, chunks,
                  chunk_units);
    launch_end(L, MOE_K_SORT_ROWS);
    return;
  }
  const size_t smem = (size_t)(p.E + 1) * 4;
  launch_begin(L, MOE_K_SORT_PLAN);
  launch_kernel(sort_count_kernel, p.nblk, kSortThreads, smem, L.stream, p);
  launch_end(L, MOE_K_SORT_PLAN);
  launch_begin(L, MOE_K_SORT_PLAN);
  launch_kernel(sort_scan_kernel, (p.E + 1 + 7) / 8, kSortThreads, 0, L.stream, p);
  launch_end(L, MOE_K_SORT_PLAN);
  launch_begin(L, MOE_K_SORT_PLAN);
  launch_kernel(sort_place_kernel, p.nblk, kSortThreads, smem, L.stream, p);
  launch_end(L, MOE_K_SORT_PLAN);
  if (!a.out) return;
  launch_begin(L, MOE_K_SORT_ROWS);
  launch_kernel(sort_rows_kernel<U>, p.T * chunks, kSortThreads, 0, L.stream, a, p.e2s, p.offsets,
                p.k, p.E, chunks, chunk_units);
  launch_end(L, MOE_K_SORT_ROWS);
}

template <typename TI, typename TO>
void launch_unsort(const Launch& L, const BackArgs& a, bool vec) {
  // slots of 128 threads; enough CTAs at any batch, each with k row loads in flight
  const int chunks = (a.nslots + 127) / 128;
  launch_begin(L, MOE_K_UNSORT);
  if (vec)
    launch_kernel(unsort_kernel<TI, TO, true>, a.T * chunks, 128, 0, L.stream, a, chunks);
  else
    launch_kernel(unsort_kernel<TI, TO, false>, a.T * chunks, 128, 0, L.stream, a, chunks);
  launch_end(L, MOE_K_UNSORT);
}

template <typename TI, typename TO>
void launch_unsort_grad(const Launch& L, GradArgs a, bool vec) {
  // few tokens: a CTA a pick, so that every SM has work
  a.picks = a.T >= 2 * L.num_sms ? a.k : 1;
  const int parts = (a.k + a.picks - 1) / a.picks;
  auto* kernel = a.drows ? (vec ? unsort_grad_kernel<TI, TO, true, true>
                                : unsort_grad_kernel<TI, TO, false, true>)
                         : (vec ? unsort_grad_kernel<TI, TO, true, false>
                                : unsort_grad_kernel<TI, TO, false, false>);
  launch_begin(L, MOE_K_UNSORT_GRAD);
  launch_kernel(kernel, a.T * parts, kGradThreads, 0, L.stream, a, parts);
  launch_end(L, MOE_K_UNSORT_GRAD);
}

// Calls f(rows type, tokens type) for a pair of float types; false if unknown.
template <typename TI, typename F>
bool with_out(int32_t out_dtype, F f) {
  switch (out_dtype) {
    case MOE_DT_BF16: f(TI{}, __nv_bfloat16{}); return true;
    case MOE_DT_FP16: f(TI{}, __half{}); return true;
    case MOE_DT_FP32: f(TI{}, 0.f); return true;
  }
  return false;
}
template <typename F>
bool with_types(int32_t dtype, int32_t out_dtype, F f) {
  switch (dtype) {
    case MOE_DT_BF16: return with_out<__nv_bfloat16>(out_dtype, f);
    case MOE_DT_FP16: return with_out<__half>(out_dtype, f);
    case MOE_DT_FP32: return with_out<float>(out_dtype, f);
  }
  return false;
}
bool is_float(int32_t dt) { return dt == MOE_DT_BF16 || dt == MOE_DT_FP16 || dt == MOE_DT_FP32; }

moe_status unsort(int32_t T, int32_t k, int32_t E, int32_t H, int32_t dtype, const void* rows,
                  const int32_t* offsets, const int32_t* e2s, const float* w, int32_t out_dtype,
                  void* out, int64_t ldo, moe_stream_t stream) {
  moe_status s = check_sort(T, k, E);
  if (s != MOE_OK) return s;
  if (H < 1 || ldo < H || !is_float(dtype) || !is_float(out_dtype)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!rows || !offsets || !e2s || !out) return MOE_ERR_INVALID_ARG;
  if (misaligned16(rows, offsets, e2s, w, out)) return MOE_ERR_ALIGNMENT;
  BackArgs a{};
  a.rows = rows;
  a.offsets = offsets;
  a.e2s = e2s;
  a.w = w;
  a.out = out;
  a.ldo = ldo;
  a.T = T;
  a.k = k;
  a.E = E;
  a.H = H;
  a.nslots = (H + kSlot - 1) / kSlot;
  if ((int64_t)T * ((a.nslots + 127) / 128) > INT_MAX) return MOE_ERR_UNSUPPORTED;
  const bool vec = H % kSlot == 0 && ldo * dtype_bytes(out_dtype) % 16 == 0;
  Launch L;
  if ((s = open_launch(stream, &L)) != MOE_OK) return s;
  with_types(dtype, out_dtype, [&](auto ti, auto to) {
    launch_unsort<decltype(ti), decltype(to)>(L, a, vec);
  });
  return launch_status_take();
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_sort_workspace_size(int32_t T, int32_t k, int32_t n_experts, size_t* bytes) {
  const moe_status s = check_sort(T, k, n_experts);
  if (s != MOE_OK) return s;
  if (!bytes) return MOE_ERR_INVALID_ARG;
  *bytes = sort_direct(T, k)
               ? 0
               : (size_t)(n_experts + 1) * block_count(T, k) * sizeof(int32_t);
  return MOE_OK;
}

moe_status moe_sort_tokens(int32_t T, int32_t k, int32_t n_experts, int32_t H, int32_t dtype,
                           const int32_t* ids, const void* x, int64_t ldx, const float* x_scale,
                           int32_t* counts, int32_t* offsets, int32_t* sorted_to_expanded,
                           int32_t* expanded_to_sorted, void* x_sorted, float* scale_sorted,
                           int32_t zero_dropped, void* ws, size_t ws_bytes, moe_stream_t stream) {
  size_t need = 0;
  moe_status s = moe_sort_workspace_size(T, k, n_experts, &need);
  if (s != MOE_OK) return s;
  const int es = dtype_bytes(dtype);
  if (zero_dropped != 0 && zero_dropped != 1) return MOE_ERR_INVALID_ARG;
  if (x_sorted && (es == 0 || H < 1 || ldx < H)) return MOE_ERR_INVALID_ARG;
  if (!counts || !offsets) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!ids || !sorted_to_expanded || !expanded_to_sorted)) return MOE_ERR_INVALID_ARG;
  if (T > 0 && x_sorted && !x) return MOE_ERR_INVALID_ARG;
  if (scale_sorted && (!x_sorted || !x_scale)) return MOE_ERR_INVALID_ARG;
  if (misaligned16(ids, x, x_scale, counts, offsets, sorted_to_expanded, expanded_to_sorted,
                   x_sorted, scale_sorted))
    return MOE_ERR_ALIGNMENT;
  if (need > 0) {
    if (!ws) return MOE_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(ws) % 256) return MOE_ERR_ALIGNMENT;
    if (ws_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  }
  PlanArgs p{};
  p.ids = ids;
  p.counts = counts;
  p.offsets = offsets;
  p.s2e = sorted_to_expanded;
  p.e2s = expanded_to_sorted;
  p.table = static_cast<int32_t*>(ws);
  p.T = T;
  p.k = k;
  p.E = n_experts;
  p.nblk = block_count(T, k);
  p.tokens = block_tokens(k);
  RowsArgs a{};
  a.x = static_cast<const unsigned char*>(x);
  a.out = static_cast<unsigned char*>(T > 0 ? x_sorted : nullptr);
  a.x_scale = x_scale;
  a.out_scale = scale_sorted;
  a.zero_dropped = zero_dropped;
  // the widest copy unit that every row of both sides is a multiple of
  const int64_t bytes = (int64_t)H * es, in_bytes = ldx * es;
  int unit = 16;
  if (a.out) {
    while (bytes % unit || (T > 1 && in_bytes % unit)) unit /= 2;
    if (bytes / unit > INT_MAX / 2) return MOE_ERR_UNSUPPORTED;
    if ((int64_t)T * row_chunks(T, (int)(bytes / unit), kSortThreads, 256) > INT_MAX / 2)
      return MOE_ERR_UNSUPPORTED;
  }
  a.ldx = in_bytes;
  a.ldo = bytes;
  a.units = a.out ? (int)(bytes / unit) : 0;
  Launch L;
  if ((s = open_launch(stream, &L)) != MOE_OK) return s;
  switch (unit) {
    case 16: launch_sort<uint4>(L, p, a); break;
    case 8: launch_sort<uint2>(L, p, a); break;
    case 4: launch_sort<uint32_t>(L, p, a); break;
    case 2: launch_sort<uint16_t>(L, p, a); break;
    default: launch_sort<uint8_t>(L, p, a); break;
  }
  return launch_status_take();
}

moe_status moe_sort_tokens_backward(int32_t T, int32_t k, int32_t n_experts, int32_t H,
                                    int32_t dtype, const void* dx_sorted, const int32_t* offsets,
                                    const int32_t* expanded_to_sorted, int32_t out_dtype, void* dx,
                                    int64_t lddx, moe_stream_t stream) {
  return unsort(T, k, n_experts, H, dtype, dx_sorted, offsets, expanded_to_sorted, nullptr,
                out_dtype, dx, lddx, stream);
}

moe_status moe_unsort_tokens(int32_t T, int32_t k, int32_t n_experts, int32_t H, int32_t dtype,
                             const void* y_sorted, const int32_t* offsets,
                             const int32_t* expanded_to_sorted, const float* topk_w,
                             int32_t out_dtype, void* out, int64_t ldo, moe_stream_t stream) {
  if (T > 0 && !topk_w) return MOE_ERR_INVALID_ARG;
  return unsort(T, k, n_experts, H, dtype, y_sorted, offsets, expanded_to_sorted, topk_w,
                out_dtype, out, ldo, stream);
}

moe_status moe_unsort_tokens_backward(int32_t T, int32_t k, int32_t n_experts, int32_t H,
                                      int32_t dtype, int32_t out_dtype, const void* dout,
                                      int64_t ldd, const void* y_sorted, const int32_t* offsets,
                                      const int32_t* expanded_to_sorted, const float* topk_w,
                                      void* dy_sorted, float* dtopk_w, int32_t zero_dropped,
                                      moe_stream_t stream) {
  moe_status s = check_sort(T, k, n_experts);
  if (s != MOE_OK) return s;
  if (H < 1 || ldd < H || !is_float(dtype) || !is_float(out_dtype)) return MOE_ERR_INVALID_ARG;
  if (zero_dropped != 0 && zero_dropped != 1) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!dout || !y_sorted || !offsets || !expanded_to_sorted || !topk_w || !dtopk_w)
    return MOE_ERR_INVALID_ARG;
  if (misaligned16(dout, y_sorted, offsets, expanded_to_sorted, topk_w, dy_sorted, dtopk_w))
    return MOE_ERR_ALIGNMENT;
  GradArgs a{};
  a.dout = dout;
  a.rows = y_sorted;
  a.offsets = offsets;
  a.e2s = expanded_to_sorted;
  a.w = topk_w;
  a.drows = dy_sorted;
  a.dw = dtopk_w;
  a.ldd = ldd;
  a.T = T;
  a.k = k;
  a.E = n_experts;
  a.H = H;
  a.nslots = (H + kSlot - 1) / kSlot;
  a.zero_dropped = zero_dropped;
  const bool vec = H % kSlot == 0 && ldd * dtype_bytes(out_dtype) % 16 == 0;
  Launch L;
  if ((s = open_launch(stream, &L)) != MOE_OK) return s;
  with_types(dtype, out_dtype, [&](auto ti, auto to) {
    launch_unsort_grad<decltype(ti), decltype(to)>(L, a, vec);
  });
  return launch_status_take();
}

}  // extern "C"
