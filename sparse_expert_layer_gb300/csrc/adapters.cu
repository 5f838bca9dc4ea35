// Low-rank adapters of many requests at once, beside a projection that they share.
//
//   v[p] = x[row p] A_j^T;   y[row p] = base[row p] + s_j v[p] B_j        (forward)
//   u[p] = s_j dy[row p] B_j^T;   dx[row p] = u[p] A_j;                   (backward)
//   dA_j = sum_p u[p]^T x[row p];   dB_j = s_j sum_p v[p]^T dy[row p]
//
// for the positions p of adapter j in the sorted order of moe_sort_tokens.  A and B lie
// as [rank][channel], so both directions are the same three products: rows times a
// matrix over its channels (shrink), a few numbers times its rows (expand), and sums
// over positions (outer).
//
// Bound by memory: the rank is small beside the channels.  Few rows: a cluster of up to
// eight CTAs takes one position from x to y, each CTA a slice of the channels on CUDA
// cores, and v is exchanged through distributed shared memory: one launch, and the
// adapters are read once.  Many rows: shrink, then expand, with rows of x and of A through
// cp.async rings into MMAs; the K of a tile of positions may be split over a cluster whose parts
// are added in order.  v, u are fp32; where they meet 16-bit factors they are split into
// two 16-bit terms (three bf16 ones for dA and dB, whose results may be fp32): 2^-17
// (bf16) or 2^-22 (fp16) of them is lost, which a rounded output does not show.
//
// Measured on a GB300, cold, us (at 6.78 TB/s): one row, rank 16, 5120 to 5120 channels 7.1 (a
// launch and three dependent reads); 64 rows of 48 adapters, 7168 to 2048 8.8 (1.6); 8192 rows,
// 5120 to 5120, rank 16 65 (37), 64 75 (39), 128 126 (40); gradients of 8192 rows, rank 16, 7168
// and 5120 channels 104 (48), rank 64, 5120 and 5120 168 (41).
#include <math.h>

#include <algorithm>

#include "mma.cuh"

namespace moe {

namespace {

constexpr int kMaxRank = 128;
constexpr int kMaxAdapters = 4096;
constexpr int kMaxCluster = 8;

struct Segments {
  const int32_t* offsets;  // [J + 1]
  const int32_t* order;    // position -> row, or nullptr
  int T, J;
  // offsets are data: stay inside the T positions whatever they hold
  __device__ __forceinline__ int at(int j) const { return min(max(offsets[j], 0), T); }
  // the row of position p, -1: none
  __device__ __forceinline__ int row(int p) const {
    const int r = order ? order[p] : p;
    return r >= 0 && r < T ? r : -1;
  }
  // the first adapter whose positions end after p, by all threads of the block
  __device__ __forceinline__ int first_after(int p) const {
    int n = 0;
    for (int j = threadIdx.x; j - (int)threadIdx.x < J; j += blockDim.x)
      n += __syncthreads_count(j < J && at(j + 1) <= p);
    return n;
  }
  // Tile `tile` when each adapter's positions (and those without one, adapter J) are cut into
  // tiles of `rows`: its adapter and positions lo .. hi.  lo >= hi: there are not so many.  By
  // all threads of the block; at most T / rows + J + 1 tiles have positions.
  __device__ __forceinline__ void tile(int index, int rows, int* adapter, int* lo, int* hi) const {
    __shared__ int sums[32], found[3];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    if (threadIdx.x == 0) found[0] = -1;
    int before = 0;
    for (int j0 = 0; j0 <= J; j0 += blockDim.x) {
      const int j = j0 + threadIdx.x;
      const int a = j <= J ? at(j) : 0, b = j < J ? at(j + 1) : T;
      const int n = j <= J && b > a ? (b - a + rows - 1) / rows : 0;
      int sum = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += up;
      }
      if (lane == 31) sums[warp] = sum;
      __syncthreads();
      int total = 0;
      for (int w = 0; w < (int)blockDim.x / 32; ++w) {
        if (w < warp) sum += sums[w];
        total += sums[w];
      }
      const int first = before + sum - n;
      if (n > 0 && index >= first && index < first + n) {
        found[0] = j;
        found[1] = a + (index - first) * rows;
        found[2] = min(b, found[1] + rows);
      }
      before += total;
      __syncthreads();
    }
    *adapter = found[0];
    *lo = found[0] >= 0 ? found[1] : 0;
    *hi = found[0] >= 0 ? found[2] : 0;
  }
  // The tiles of the adapters before j, by all threads of the block.
  __device__ __forceinline__ int tiles_before(int j, int rows) const {
    __shared__ int parts[32];
    int n = 0;
    for (int i = threadIdx.x; i < j; i += blockDim.x)
      n += (max(0, at(i + 1) - at(i)) + rows - 1) / rows;
    n = __reduce_add_sync(0xffffffffu, n);
    if (threadIdx.x % 32 == 0) parts[threadIdx.x / 32] = n;
    __syncthreads();
    n = 0;
    for (int w = 0; w < (int)blockDim.x / 32; ++w) n += parts[w];
    return n;
  }
};

__device__ __forceinline__ void sts128(uint32_t at, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}
// Piece i (channels 8 i ..) of a row of n channels, zeros past its end.
template <typename T>
__device__ __forceinline__ uint4 load_piece(const T* row, int i, int n, bool vec) {
  if (vec) return 8 * i < n ? *reinterpret_cast<const uint4*>(row + 8 * i) : make_uint4(0u, 0u, 0u, 0u);
  T v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = 8 * i + j < n ? row[8 * i + j] : from_f<T>(0.f);
  uint4 q;
  memcpy(&q, v, 16);
  return q;
}
template <typename T>
__device__ __forceinline__ void unpack_piece(const uint4& q, float (&f)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = unpack2<T>(w[i]);
    f[2 * i] = v.x;
    f[2 * i + 1] = v.y;
  }
}
template <typename T>
__device__ __forceinline__ void store_words(T* row, int i, int n, bool vec, const uint4& q) {
  if (vec) {
    if (8 * i < n) *reinterpret_cast<uint4*>(row + 8 * i) = q;
    return;
  }
  T v[8];
  memcpy(v, &q, 16);
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (8 * i + j < n) row[8 * i + j] = v[j];
}
template <typename T>
__device__ __forceinline__ void store_piece(T* row, int i, int n, bool vec, const float (&f)[8]) {
  store_words<T>(row, i, n, vec, pack8<T>(f).q[0]);
}
// The same into shared memory: asynchronous where rows are whole pieces.
template <typename T>
__device__ __forceinline__ void stage_piece(uint32_t dst, const T* row, int i, int n, bool vec,
                                            bool real) {
  if (vec) {
    const bool in = real && 8 * i < n;
    cp_async16_or_zero(dst, row + (in ? 8 * i : 0), in);
  } else {
    sts128(dst, real ? load_piece<T>(row, i, n, false) : make_uint4(0u, 0u, 0u, 0u));
  }
}

__device__ __forceinline__ void ldsm4(uint32_t at, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}

// The largest |v| that a block has seen, for the range of fp16 terms: one word a block.
__device__ __forceinline__ uint32_t block_max(uint32_t bits) {
  __shared__ uint32_t most[32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) bits = max(bits, __shfl_xor_sync(0xffffffffu, bits, o));
  __syncthreads();
  if (threadIdx.x % 32 == 0) most[threadIdx.x / 32] = bits;
  __syncthreads();
  for (int i = 0; i < (int)blockDim.x / 32; ++i) bits = max(bits, most[i]);
  return bits;
}

struct AdapterArgs {
  Segments seg;
  const void* x;  // shrink: rows [T, K] times m1 [J, r, K]
  int64_t ldx;
  const void* m1;
  const float* scale1;  // of v, or nullptr
  float* v;             // [T, r], by position
  const void* m2;       // expand: v times m2 [J, r, N]
  const float* scale2;
  const void* base;     // [T, N], or nullptr: zeros
  int64_t ldb;
  void* y;
  int64_t ldy;
  const float* other;   // backward: the v of the forward pass
  uint32_t* max_v;      // backward: largest |v|, |other| of each block
  uint32_t* max_other;
  int r, K, N;
  int xvec, m1vec, m2vec, yvec;
};

// ---------------------------------------------------------------- few rows ----
constexpr int kRowSide = 128;  // threads side by side along the second product's columns

// One position: a cluster's CTAs take slices of K, then slices of N.  A warp takes four ranks of
// the first product at once, 128 threads eight of the second: more WARPS, fewer dependent reads.
template <typename T, int WARPS>
__global__ void __launch_bounds__(32 * WARPS) adapters_row_kernel(AdapterArgs a) {
  constexpr int kThreads = 32 * WARPS, kGroups = kThreads / kRowSide;
  __shared__ float red[kGroups > 1 ? (kGroups - 1) * 8 * kRowSide : 1];
  pdl_enter();
  __shared__ float part[kMaxRank], total[kMaxRank];
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int rank = blockIdx.x, C = gridDim.x, p = blockIdx.y, r = a.r;
  const int j = a.seg.first_after(p);
  const int row = a.seg.row(p);
  const bool has = j < a.seg.J && a.seg.at(j) <= p && row >= 0;
  const int n8 = (a.N + 7) / 8, np = (n8 + C - 1) / C;
  const int n0 = min(n8, rank * np), n1 = min(n8, n0 + np);
  T* yrow = static_cast<T*>(a.y) + row * a.ldy;
  const T* brow = a.base ? static_cast<const T*>(a.base) + row * a.ldb : nullptr;
  if (!has) {  // the whole cluster; the row is its base
    if (row >= 0 && a.y != a.base)
      for (int i = n0 + tid; i < n1; i += kThreads) {
        float f[8] = {};
        if (brow) unpack_piece<T>(load_piece<T>(brow, i, a.N, a.yvec), f);
        store_piece<T>(yrow, i, a.N, a.yvec, f);
      }
    if (rank == 0 && row < 0 && j < a.seg.J && a.seg.at(j) <= p)
      for (int i = tid; i < r; i += kThreads) a.v[(int64_t)p * r + i] = 0.f;
    if (a.max_v && tid == 0) {
      a.max_v[p * C + rank] = 0u;
      a.max_other[p * C + rank] = 0u;
    }
    return;
  }
  const T* m2 = static_cast<const T*>(a.m2) + (int64_t)j * r * a.N;
  // the second matrix's slice on its way to L2 while the first is read
  if (a.y && a.m2vec)
    for (int i = tid; i < r * (n1 - n0); i += kThreads)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(m2 + (int64_t)(i / (n1 - n0)) * a.N +
                                                    8 * (n0 + i % (n1 - n0))));
  const T* xrow = static_cast<const T*>(a.x) + row * a.ldx;
  const T* m1 = static_cast<const T*>(a.m1) + (int64_t)j * r * a.K;
  const int k8 = (a.K + 7) / 8, kp = (k8 + C - 1) / C;
  const int k0 = min(k8, rank * kp), k1 = min(k8, k0 + kp);
  constexpr int kRanks = 4, kAtOnce = 4;  // ranks of a warp, pieces of a lane in flight
  for (int i0 = warp * kRanks; i0 < r; i0 += WARPS * kRanks) {
    float acc[kRanks] = {};
    for (int kb = k0; kb < k1; kb += 32 * kAtOnce) {
      uint4 xq[kAtOnce], mq[kAtOnce][kRanks];
#pragma unroll
      for (int q = 0; q < kAtOnce; ++q) {
        const int k = kb + q * 32 + lane;
        const uint4 none = make_uint4(0u, 0u, 0u, 0u);
        xq[q] = k < k1 ? load_piece<T>(xrow, k, a.K, a.xvec) : none;
#pragma unroll
        for (int i = 0; i < kRanks; ++i)
          mq[q][i] = k < k1 && i0 + i < r
                         ? load_piece<T>(m1 + (int64_t)(i0 + i) * a.K, k, a.K, a.m1vec)
                         : none;
      }
#pragma unroll
      for (int q = 0; q < kAtOnce; ++q) {
        float xf[8], mf[8];
        unpack_piece<T>(xq[q], xf);
#pragma unroll
        for (int i = 0; i < kRanks; ++i) {
          unpack_piece<T>(mq[q][i], mf);
#pragma unroll
          for (int c = 0; c < 8; ++c) acc[i] = fmaf(xf[c], mf[c], acc[i]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kRanks; ++i) {
      const float s = warp_sum(acc[i]);
      if (lane == 0 && i0 + i < r) part[i0 + i] = s;
    }
  }
  cluster_sync_all();
  const float s1 = a.scale1 ? a.scale1[j] : 1.f, s2 = a.scale2 ? a.scale2[j] : 1.f;
  uint32_t most = 0u, most_other = 0u;
  for (int i = tid; i < r; i += kThreads) {
    float s = 0.f;
    for (int q = 0; q < C; ++q) s += ld_cluster_f32(mapa_shared(smem_u32(&part[i]), q));
    s *= s1;
    total[i] = s;
    if (rank == 0) {
      a.v[(int64_t)p * r + i] = s;
      most = max(most, magnitude(s));
      if (a.other) most_other = max(most_other, magnitude(a.other[(int64_t)p * r + i]));
    }
  }
  if (a.max_v) {
    most = block_max(most);
    most_other = block_max(most_other);
    if (tid == 0) {
      a.max_v[p * C + rank] = most;
      a.max_other[p * C + rank] = most_other;
    }
  }
  __syncthreads();
  // (no CTA leaves while another reads its part: waited for at the end)
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  // a thread has eight columns and adds up the ranks of its group
  const int group = tid / kRowSide, side = tid % kRowSide;
  for (int i0 = n0; i0 < n1 && a.y; i0 += kRowSide) {
    const int i = i0 + side;
    const bool in = i < n1;
    float f[8] = {}, acc[8] = {};
    const uint4 bq = brow && in && group == 0 ? load_piece<T>(brow, i, a.N, a.yvec)
                                              : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 1
    for (int q0 = 8 * group; q0 < r && in; q0 += 8 * kGroups) {
      uint4 mq[8];
#pragma unroll
      for (int q = 0; q < 8; ++q)
        mq[q] = q0 + q < r ? load_piece<T>(m2 + (int64_t)(q0 + q) * a.N, i, a.N, a.m2vec)
                           : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        float m[8];
        unpack_piece<T>(mq[q], m);
        const float v = q0 + q < r ? total[q0 + q] : 0.f;
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[c] = fmaf(v, m[c], acc[c]);
      }
    }
    if constexpr (kGroups > 1) {  // the groups' parts, added in order
      if (group > 0) {
#pragma unroll
        for (int c = 0; c < 8; ++c) red[((group - 1) * 8 + c) * kRowSide + side] = acc[c];
      }
      __syncthreads();
      if (group == 0) {
#pragma unroll
        for (int q = 0; q < kGroups - 1; ++q)
#pragma unroll
          for (int c = 0; c < 8; ++c) acc[c] += red[(q * 8 + c) * kRowSide + side];
      }
    }
    if (group == 0 && in) {
      unpack_piece<T>(bq, f);
#pragma unroll
      for (int c = 0; c < 8; ++c) f[c] = fmaf(s2, acc[c], f[c]);
      store_piece<T>(yrow, i, a.N, a.yvec, f);
    }
    if constexpr (kGroups > 1) __syncthreads();
  }
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// ------------------------------------------------------------------ shrink ----
constexpr int kShrinkStages = 4;
// positions of a tile: more where the adapter's rows are many beside them
template <int RT>
constexpr int kShrinkRows = RT <= 32 ? 64 : 128;
int shrink_rows(int r) { return r <= 32 ? 64 : 128; }

// v of a tile of one adapter's positions: x rows and the adapter's rows in 128-byte slices of
// K.  Slice c of row i lies at 16-byte piece c ^ (i % 8), so that neither copies nor ldmatrix
// meet a bank twice.  A warp has 16 positions and all ranks.  Waits for slices: 3.7 TB/s at rank
// 16 (8192 rows of 5120, 23 us), 2.8 at rank 64 (32 us; shared memory half busy).
template <typename T, int RT>
__global__ void __launch_bounds__(2 * kShrinkRows<RT>) adapters_shrink_kernel(AdapterArgs a) {
  pdl_enter();
  extern __shared__ __align__(128) unsigned char smem[];
  constexpr int kRows = kShrinkRows<RT>, kThreads = 2 * kRows;
  constexpr int kX = kRows * 128, kStage = kX + RT * 128;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int rank = blockIdx.x, S = gridDim.x, r = a.r;
  const uint32_t base = smem_u32(smem);
  int j, lo, hi;
  a.seg.tile(blockIdx.y, kRows, &j, &lo, &hi);
  if (lo >= hi || j >= a.seg.J) {  // the whole cluster
    if (a.max_v && tid == 0) a.max_v[blockIdx.y * S + rank] = a.max_other[blockIdx.y * S + rank] = 0u;
    return;
  }
  const int slices = (a.K + 63) / 64;
  const int c0 = (int)((int64_t)slices * rank / S), c1 = (int)((int64_t)slices * (rank + 1) / S);
  constexpr int kStep = kThreads / 8;  // rows that the threads copy at once
  const int piece = tid % 8;
  const T* xr[kRows / kStep];
  bool real[kRows / kStep];
#pragma unroll
  for (int i = 0; i < kRows / kStep; ++i) {
    const int p = lo + tid / 8 + kStep * i;
    const int row = p < hi ? a.seg.row(p) : -1;
    real[i] = row >= 0;
    xr[i] = static_cast<const T*>(a.x) + (real[i] ? row * a.ldx : 0);
  }
  const T* m = static_cast<const T*>(a.m1) + ((int64_t)j * r) * a.K;
  auto load = [&](int c, int slot) {
    const uint32_t st = base + slot * kStage;
#pragma unroll
    for (int i = 0; i < kRows / kStep; ++i) {
      const int row = tid / 8 + kStep * i;
      stage_piece<T>(st + row * 128 + ((piece ^ (row % 8)) * 16), xr[i], c * 8 + piece, a.K, a.xvec,
                     real[i]);
    }
#pragma unroll
    for (int i = 0; i < (RT + kStep - 1) / kStep; ++i) {
      const int row = tid / 8 + kStep * i;
      const bool in = row < r;
      if (row < RT)
        stage_piece<T>(st + kX + row * 128 + ((piece ^ (row % 8)) * 16),
                       m + (in ? (int64_t)row * a.K : 0), c * 8 + piece, a.K, a.m1vec, in);
    }
  };
  // MMAs cut their sums off where fp32 ends, each time the same way: after every kFlush slices
  // (sixteen MMAs) what they hold is added, rounded, to the sum.
  constexpr int kFlush = 4;
  float acc[RT / 8][4] = {}, sum[RT / 8][4] = {};
  auto flush = [&]() {
#pragma unroll
    for (int n = 0; n < RT / 8; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sum[n][i] += acc[n][i];
        acc[n][i] = 0.f;
      }
  };
#pragma unroll
  for (int q = 0; q < kShrinkStages - 1; ++q) {
    if (c0 + q < c1) load(c0 + q, q);
    cp_async_commit();
  }
  for (int c = c0; c < c1; ++c) {
    cp_async_wait<kShrinkStages - 2>();
    __syncthreads();
    const int ahead = c + kShrinkStages - 1;
    if (ahead < c1) load(ahead, (ahead - c0) % kShrinkStages);
    cp_async_commit();
    const uint32_t st = base + (c - c0) % kShrinkStages * kStage;
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      uint32_t af[4];
      const int row = warp * 16 + lane % 16;
      ldsm4(st + row * 128 + (((kk * 2 + lane / 16) ^ (row % 8)) * 16), af);
#pragma unroll
      for (int n = 0; n < RT / 16; ++n) {
        uint32_t bf[4];
        const int i = n * 16 + lane % 8 + lane / 16 * 8;
        ldsm4(st + kX + i * 128 + (((kk * 2 + lane / 8 % 2) ^ (i % 8)) * 16), bf);
        mma16816<T>(acc[2 * n], af[0], af[1], af[2], af[3], bf[0], bf[1]);
        mma16816<T>(acc[2 * n + 1], af[0], af[1], af[2], af[3], bf[2], bf[3]);
      }
    }
    if ((c - c0) % kFlush == kFlush - 1) flush();
  }
  flush();
  cp_async_wait<0>();
  __syncthreads();
  float* red = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int n = 0; n < RT / 8; ++n) {
    float* at = red + (warp * 16 + lane / 4) * RT + n * 8 + lane % 4 * 2;
    *reinterpret_cast<float2*>(at) = make_float2(sum[n][0], sum[n][1]);
    *reinterpret_cast<float2*>(at + 8 * RT) = make_float2(sum[n][2], sum[n][3]);
  }
  cluster_sync_all();
  const float s1 = a.scale1 ? a.scale1[j] : 1.f;
  uint32_t most = 0u;
  for (int e = rank * kThreads + tid; e < kRows * RT; e += S * kThreads) {
    const int p = lo + e / RT, i = e % RT;
    if (p >= hi || i >= r) continue;
    float s = 0.f;
    for (int q = 0; q < S; ++q) s += ld_cluster_f32(mapa_shared(base + e * 4, q));
    s *= s1;
    a.v[(int64_t)p * r + i] = s;
    most = max(most, magnitude(s));
  }
  cluster_sync_all();
  if (a.max_v) {
    uint32_t other = 0u;
    for (int64_t i = (int64_t)lo * r + rank * kThreads + tid; i < (int64_t)hi * r; i += S * kThreads)
      other = max(other, magnitude(a.other[i]));
    most = block_max(most);
    other = block_max(other);
    if (tid == 0) {
      a.max_v[blockIdx.y * S + rank] = most;
      a.max_other[blockIdx.y * S + rank] = other;
    }
  }
}

// The same for more than 64 ranks through tcgen05, whose operands the slices are as they lie: M is
// the 128 positions, N the ranks, accumulators in tensor memory.  A thread issues a slice's MMAs,
// their completion frees its stage.  Two accumulators in turn: while one has the MMAs of kFlush
// slices, what the other holds is added, rounded, to sums in registers, as above.  Of ldmatrix and
// mma.sync 128 ranks are too many: 8192 rows of 5120 to 5120 in 154 us, here 130; of 64 ranks the
// call takes 75 us with those and 86 with this.
template <typename T, int RT>
__global__ void __launch_bounds__(256, RT <= 64 ? 2 : 1) adapters_shrink_tc_kernel(AdapterArgs a) {
  extern __shared__ unsigned char raw[];
  __shared__ uint64_t bars[kShrinkStages];
  __shared__ uint32_t tmem_slot;
  constexpr int kRows = 128, kThreads = 256;
  constexpr int kX = kRows * 128, kStage = kX + RT * 128;
  constexpr int kAccums = 2, kFlush = 4;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int rank = blockIdx.x, S = gridDim.x, r = a.r;
  // (the same offset in every CTA of the cluster)
  const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
  pdl_wait();
  int j, lo, hi;
  a.seg.tile(blockIdx.y, kRows, &j, &lo, &hi);
  if (lo >= hi || j >= a.seg.J) {  // the whole cluster
    if (a.max_v && tid == 0) a.max_v[blockIdx.y * S + rank] = a.max_other[blockIdx.y * S + rank] = 0u;
    return;
  }
  const int slices = (a.K + 63) / 64;
  const int c0 = (int)((int64_t)slices * rank / S), c1 = (int)((int64_t)slices * (rank + 1) / S);
  constexpr int kStep = kThreads / 8;  // rows that the threads copy at once
  const int piece = tid % 8;
  const T* xr[kRows / kStep];
  bool real[kRows / kStep];
#pragma unroll
  for (int i = 0; i < kRows / kStep; ++i) {
    const int p = lo + tid / 8 + kStep * i;
    const int row = p < hi ? a.seg.row(p) : -1;
    real[i] = row >= 0;
    xr[i] = static_cast<const T*>(a.x) + (real[i] ? row * a.ldx : 0);
  }
  const T* m = static_cast<const T*>(a.m1) + ((int64_t)j * r) * a.K;
  auto load = [&](int c, int slot) {
    const uint32_t st = base + slot * kStage;
#pragma unroll
    for (int i = 0; i < kRows / kStep; ++i) {
      const int row = tid / 8 + kStep * i;
      stage_piece<T>(st + row * 128 + ((piece ^ (row % 8)) * 16), xr[i], c * 8 + piece, a.K, a.xvec,
                     real[i]);
    }
#pragma unroll
    for (int i = 0; i < RT / kStep; ++i) {
      const int row = tid / 8 + kStep * i;
      const bool in = row < r;
      stage_piece<T>(st + kX + row * 128 + ((piece ^ (row % 8)) * 16),
                     m + (in ? (int64_t)row * a.K : 0), c * 8 + piece, a.K, a.m1vec, in);
    }
  };
#pragma unroll
  for (int q = 0; q < kShrinkStages - 1; ++q) {
    if (c0 + q < c1) load(c0 + q, q);
    cp_async_commit();
  }
  if (tid == 0) {
#pragma unroll
    for (int q = 0; q < kShrinkStages; ++q) mbar_init(smem_u32(&bars[q]), 1);
    fence_barrier_init();
  }
  __syncwarp();
  if (warp == 0) tmem_alloc(smem_u32(&tmem_slot), kAccums * RT);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();  // (as in the expand: after every CTA has its tensor memory)
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&tmem_slot);
  const uint32_t idesc = std::is_same<T, __half>::value ? idesc_f16_f32(kRows, RT)
                                                        : idesc_bf16_f32(kRows, RT);
  // a warp has 32 positions, a lane one of them, and half the ranks
  float sum[RT / 64][32] = {};
  auto flush = [&](int chunk) {
    tc_fence_after();
#pragma unroll
    for (int h = 0; h < RT / 64; ++h) {
      uint32_t d[32];
      tmem_ld32(tmem + ((uint32_t)(warp % 4 * 32) << 16) + chunk % kAccums * RT +
                    warp / 4 * (RT / 2) + 32 * h, d);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 32; ++i) sum[h][i] += __uint_as_float(d[i]);
    }
    tc_fence_before();
  };
  bool ok = true;
  for (int c = c0; c < c1; ++c) {
    const int n = c - c0, slot = n % kShrinkStages;
    cp_async_wait<kShrinkStages - 2>();
    fence_proxy_async_smem();
    __syncthreads();
    if (tid == 0) {
      tc_fence_after();
      const uint32_t st = base + slot * kStage;
      const uint32_t d = tmem + n / kFlush % kAccums * RT;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        tc_mma_bf16(d, sdesc_sw128(st + k * 32), sdesc_sw128(st + kX + k * 32), idesc,
                    n % kFlush > 0 || k > 0);
      tc_commit(smem_u32(&bars[slot]));
    }
    __syncwarp();
    // the stage of the slice before is free when its MMAs are done, and so are its accumulator's
    const int ahead = c + kShrinkStages - 1;
    if (n > 0) ok = warp_wait(smem_u32(&bars[(n - 1) % kShrinkStages]),
                              (n - 1) / kShrinkStages & 1) && ok;
    if (ahead < c1) load(ahead, (ahead - c0) % kShrinkStages);
    cp_async_commit();
    if (n > 0 && n % kFlush == 0) flush(n / kFlush - 1);
  }
  const int all = c1 - c0;
  if (all > 0) {
    ok = warp_wait(smem_u32(&bars[(all - 1) % kShrinkStages]), (all - 1) / kShrinkStages & 1) && ok;
    flush((all - 1) / kFlush);
  }
  cp_async_wait<0>();
  __syncthreads();
  // [position][rank]; (rows of 33 x 4 bytes would be out of step with the other CTAs': turn the
  // columns instead)
  float* red = reinterpret_cast<float*>(raw + (base - smem_u32(raw)));
  float* at = red + (warp % 4 * 32 + lane) * RT;
#pragma unroll
  for (int h = 0; h < RT / 64; ++h)
#pragma unroll
    for (int i = 0; i < 32; ++i)
      at[(warp / 4 * (RT / 2) + 32 * h + i) ^ lane] = ok ? sum[h][i] : NAN;
  tc_fence_before();
  cluster_sync_all();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kAccums * RT);
  }
  const float s1 = a.scale1 ? a.scale1[j] : 1.f;
  uint32_t most = 0u;
  for (int e = rank * kThreads + tid; e < kRows * RT; e += S * kThreads) {
    const int row = e / RT, i = e % RT, p = lo + row;
    if (p >= hi || i >= r) continue;
    float s = 0.f;
    for (int q = 0; q < S; ++q)
      s += ld_cluster_f32(mapa_shared(base + (row * RT + (i ^ (row % 32))) * 4, q));
    s *= s1;
    a.v[(int64_t)p * r + i] = s;
    most = max(most, magnitude(s));
  }
  cluster_sync_all();
  if (a.max_v) {
    uint32_t other = 0u;
    for (int64_t i = (int64_t)lo * r + rank * kThreads + tid; i < (int64_t)hi * r; i += S * kThreads)
      other = max(other, magnitude(a.other[i]));
    most = block_max(most);
    other = block_max(other);
    if (tid == 0) {
      a.max_v[blockIdx.y * S + rank] = most;
      a.max_other[blockIdx.y * S + rank] = other;
    }
  }
}

// ------------------------------------------------------------------ expand ----
constexpr int kExpandRows = 128;
constexpr int kExpandThreads = 256;
template <int RT>
constexpr int kExpandPerSm = RT <= 64 ? 2 : 1;  // CTAs
constexpr int kExpandTile = 128;  // columns of an accumulator, one of two
constexpr uint32_t kExpandTmem = 2 * kExpandTile;

// Sixteen lanes x 32 columns of fp32: a lane has columns 8 i + 2 (lane % 4) and the next of rows
// lane / 4 (r[4 i], r[4 i + 1]) and lane / 4 + 8 (r[4 i + 2], r[4 i + 3]).
__device__ __forceinline__ void tmem_ld_rows(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// An MMA's operand whose rows (of K) have their elements of M or N side by side: 64 of them are 128
// bytes, eight rows an atom of the 128-byte swizzle, `chunk` bytes to the next 64 elements.
__device__ __forceinline__ uint64_t sdesc_rows(uint32_t at, uint32_t chunk) {
  return sdesc_sw128(at) - ((uint64_t)1u << 16) + ((uint64_t)(chunk >> 4) << 16);
}

// y of a tile of one adapter's positions and a range of columns through tcgen05: v as two terms of
// 16 bits in shared memory, times tiles of 128 columns of the second matrix, into one of two
// accumulators while the other is read.  A warp has 32 positions and 64 columns of a tile; the
// columns of 32 are dealt to the accumulator so that a lane's results are eight neighbours of a
// position: pair t of 16-byte piece q lies at columns 8 t + 2 q and the next.  The base of the
// next tile is in registers.
// LINES (base and at most 32 ranks): 8192 rows, 5120 to 5120, rank 16 65 us and 73 without, rank
// 32 70 and 77; rank 64 77 and 75, and without a base 109 and 107 (gradients of 8192 rows).  Through
// shared memory, a position a lane: 66 and 78 (ranks 16, 64), gradients 120; a lane writing 64
// columns of a position itself 89 and 81.  With mma.sync and v in registers the same calls took 79
// and 85, gradients 111.
template <typename T, int RT, bool LINES>
__global__ void __launch_bounds__(kExpandThreads, kExpandPerSm<RT>)
    adapters_expand_kernel(AdapterArgs a, int range) {
  extern __shared__ unsigned char raw[];
  __shared__ uint64_t bars[2];
  __shared__ uint32_t tmem_slot;
  __shared__ float row_scale[kExpandRows];
  constexpr bool kHalf = std::is_same<T, __half>::value;
  constexpr int kAtoms = (RT + 63) / 64, kTerm = kAtoms * kExpandRows * 128;  // bytes of a term
  constexpr int kChunk = RT * 128, kTile = kExpandTile / 64 * kChunk;
  const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
  const uint32_t tiles = base + 2 * kTerm;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int r = a.r, n_begin = blockIdx.x * range, n_end = min(a.N, n_begin + range);
  // (what the kernel before does not write is read before the wait for it: that kernel let this
  // one start only after its own)
  int j, lo, hi;
  a.seg.tile(blockIdx.y, kExpandRows, &j, &lo, &hi);
  if (lo >= hi || j >= a.seg.J) pdl_wait();  // no CTA ends before the kernel before has
  if (lo >= hi) return;
  if (j >= a.seg.J) {  // rows without an adapter are their base
    if (a.y == a.base) return;
    for (int p = lo + warp; p < hi; p += kExpandThreads / 32) {
      const int row = a.seg.row(p);
      if (row < 0) continue;
      for (int i = n_begin / 8 + lane; 8 * i < n_end; i += 32) {
        float f[8] = {};
        if (a.base)
          unpack_piece<T>(
              load_piece<T>(static_cast<const T*>(a.base) + row * a.ldb, i, a.N, a.yvec), f);
        store_piece<T>(static_cast<T*>(a.y) + row * a.ldy, i, a.N, a.yvec, f);
      }
    }
    return;
  }
  const T* m = static_cast<const T*>(a.m2) + (int64_t)j * r * a.N;
  auto load_tile = [&](int n0, int buf) {
    constexpr int kWords = kExpandTile / 2;
#pragma unroll
    for (int e0 = 0; e0 < RT * kWords; e0 += kExpandThreads) {
      const int e = e0 + tid, i = e / kWords, w = e % kWords, t = w % 4, q = w / 4 % 4;
      const int n = n0 + 2 * w;
      const uint32_t dst = tiles + buf * kTile + w / 32 * kChunk + i * 128 +
                           (((w / 16 % 2 * 4 + t) ^ (i % 8)) * 16) + 4 * q;
      const T* from = m + (int64_t)i * a.N + n;
      if (i < r && n < a.N && a.m2vec) {
        cp_async_unit(dst, from, 4);
      } else {
        T v[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) v[c] = i < r && n + c < a.N ? from[c] : from_f<T>(0.f);
        uint32_t pair;
        memcpy(&pair, v, 4);
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(dst), "r"(pair) : "memory");
      }
    }
  };
  load_tile(n_begin, 0);
  cp_async_commit();
  if (n_begin + kExpandTile < n_end) load_tile(n_begin + kExpandTile, 1);
  cp_async_commit();
  if (tid == 0) {
    mbar_init(smem_u32(&bars[0]), 1);
    mbar_init(smem_u32(&bars[1]), 1);
    fence_barrier_init();
  }
  // The lane's four positions are mine + 8 i, and two pieces of each: tg and tg + 4 of a line of 64
  // columns.  LINES: lanes with the positions beside them (lane ^ 4) pass half of the even one's
  // line and then half of the odd one's, so that eight lanes read and write whole lines.
  const int mine = warp % 4 * 32 + lane / 4, col = warp / 4 * 64, tg = lane % 4;
  const bool odd = lane & 4;
  int row[4][2];
  bool any = false;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int p = lo + (LINES ? (mine & ~1) + q : mine) + 8 * i;
      row[i][q] = p < hi ? a.seg.row(p) : -1;
      any = any || row[i][q] >= 0;
    }
  any = __any_sync(0xffffffffu, any);
  auto piece = [&](int q) { return tg + (LINES ? (odd ? 4 : 0) : 4 * q); };
  uint4 next[4][2];
  auto load_base = [&](int n, int i, int q) {
    next[i][q] = make_uint4(0u, 0u, 0u, 0u);
    if (a.base && row[i][q] >= 0 && n + 8 * piece(q) < n_end)
      next[i][q] = load_piece<T>(static_cast<const T*>(a.base) + row[i][q] * a.ldb,
                                 n / 8 + piece(q), a.N, a.yvec);
  };
  // (even, odd) rows' pieces <-> the own position's pieces tg and tg + 4
  auto swap_halves = [&](uint4& even, uint4& other) {
    const uint4 give = odd ? even : other;
    uint4 got;
    got.x = __shfl_xor_sync(0xffffffffu, give.x, 4);
    got.y = __shfl_xor_sync(0xffffffffu, give.y, 4);
    got.z = __shfl_xor_sync(0xffffffffu, give.z, 4);
    got.w = __shfl_xor_sync(0xffffffffu, give.w, 4);
    if (odd)
      even = got;
    else
      other = got;
  };
#pragma unroll
  for (int i = 0; i < 8; ++i) load_base(n_begin + col, i % 4, i / 4);
  // (no kernel that waits for this one starts, and takes tensor memory, before every CTA of this
  // one has its own)
  __syncwarp();
  if (warp == 0) tmem_alloc(smem_u32(&tmem_slot), kExpandTmem);
  pdl_wait();
  // v as two terms: a row's pieces of eight ranks by neighbouring lanes
  {
    const float scale = a.scale2 ? a.scale2[j] : 1.f;
    constexpr int kRowLanes = RT / 8;
#pragma unroll
    for (int e0 = 0; e0 < kExpandRows * kRowLanes; e0 += kExpandThreads) {
      const int e = e0 + tid, i = e / kRowLanes, k8 = e % kRowLanes;
      const bool in = lo + i < hi;
      const float* v = a.v + (int64_t)(lo + (in ? i : 0)) * r;
      float f[8] = {};
      if (r % 8 == 0) {
        if (in && k8 * 8 < r) {
          *reinterpret_cast<float4*>(f) = *reinterpret_cast<const float4*>(v + k8 * 8);
          *reinterpret_cast<float4*>(f + 4) = *reinterpret_cast<const float4*>(v + k8 * 8 + 4);
        }
      } else {
#pragma unroll
        for (int c = 0; c < 8; ++c)
          if (in && k8 * 8 + c < r) f[c] = v[k8 * 8 + c];
      }
      float up = scale;  // bf16: scale * v
      if constexpr (kHalf) {  // into fp16's range, row by row; scaled back afterwards
        uint32_t most = 0u;
#pragma unroll
        for (int c = 0; c < 8; ++c) most = max(most, magnitude(f[c]));
#pragma unroll
        for (int o = 1; o < kRowLanes; o <<= 1)
          most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
        const uint32_t bits = fp16_range_bits(most);
        up = __uint_as_float(bits);
        if (k8 == 0) row_scale[i] = scale * inverse_pow2(bits);
      }
      uint32_t first[4], rest[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) split2<T>(f[2 * c] * up, f[2 * c + 1] * up, first[c], rest[c]);
      const uint32_t at =
          base + k8 / 8 * (kExpandRows * 128) + i * 128 + (((k8 % 8) ^ (i % 8)) * 16);
      sts128(at, make_uint4(first[0], first[1], first[2], first[3]));
      sts128(at + kTerm, make_uint4(rest[0], rest[1], rest[2], rest[3]));
    }
  }
  cp_async_wait<1>();
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&tmem_slot);
  const uint32_t idesc = (kHalf ? idesc_f16_f32(kExpandRows, kExpandTile)
                                : idesc_bf16_f32(kExpandRows, kExpandTile)) |
                         (1u << 16);  // B's columns side by side
  auto multiply = [&](int buf) {  // one thread
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int k = 0; k < RT / 16; ++k)
        tc_mma_bf16(tmem + buf * kExpandTile,
                    sdesc_sw128(base + t * kTerm + k / 4 * (kExpandRows * 128) + k % 4 * 32),
                    sdesc_rows(tiles + buf * kTile + k * 2048, kChunk), idesc, t > 0 || k > 0);
    tc_commit(smem_u32(&bars[buf]));
  };
  if (tid == 0) multiply(0);
  float back[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) back[i] = kHalf ? row_scale[mine + 8 * i] : 1.f;
  int use = 0;
  for (int n0 = n_begin; n0 < n_end; n0 += kExpandTile, ++use) {
    const int buf = use & 1;
    const bool more = n0 + kExpandTile < n_end;
    if (more) {  // the next tile is there, and nobody reads its accumulator
      cp_async_wait<0>();
      fence_proxy_async_smem();
      tc_fence_before();
      __syncthreads();
      tc_fence_after();
      if (tid == 0) multiply(buf ^ 1);
      __syncwarp();
    }
    if (!warp_wait(smem_u32(&bars[buf]), (use >> 1) & 1))  // gave up: no numbers then
      back[0] = back[1] = back[2] = back[3] = NAN;
    tc_fence_after();
    if (n0 + 2 * kExpandTile < n_end) load_tile(n0 + 2 * kExpandTile, buf);
    cp_async_commit();
    if (!any) continue;
    const int n = n0 + col;
    // a piece of position i: base plus its part of 16 positions and 32 columns
    auto finish = [&](uint4 base, const uint32_t (&d)[16], int i) {
      float f[8] = {};
      if (a.base) unpack_piece<T>(base, f);
#pragma unroll
      for (int c = 0; c < 8; ++c)
        f[c] = fmaf(back[i], __uint_as_float(d[c / 2 * 4 + i % 2 * 2 + c % 2]), f[c]);
      return pack8<T>(f).q[0];
    };
    auto store = [&](int i, int q, const uint4& v) {
      if (row[i][q] >= 0 && n + 8 * piece(q) < n_end)
        store_words<T>(static_cast<T*>(a.y) + row[i][q] * a.ldy, n / 8 + piece(q), a.N, a.yvec, v);
      load_base(n + kExpandTile, i, q);
    };
    const uint32_t acc = tmem + ((uint32_t)(warp % 4 * 32) << 16) + buf * kExpandTile + col;
#pragma unroll
    for (int k = 0; k < 2; ++k) {  // 16 positions of a line, or 32 of half of one
      uint32_t d[2][16];
#pragma unroll
      for (int l = 0; l < 2; ++l)
        tmem_ld_rows(acc + ((uint32_t)(16 * (LINES ? k : l)) << 16) + 32 * (LINES ? l : k), d[l]);
      tmem_ld_wait();
      if constexpr (LINES) {
#pragma unroll
        for (int i = 2 * k; i < 2 * k + 2; ++i) {
          uint4 q0 = next[i][0], q1 = next[i][1];
          swap_halves(q0, q1);
          q0 = finish(q0, d[0], i);
          q1 = finish(q1, d[1], i);
          swap_halves(q0, q1);
          store(i, 0, q0);
          store(i, 1, q1);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) store(i, k, finish(next[i][k], d[i / 2], i));
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kExpandTmem);
  }
}

// ------------------------------------------------------------------- outer ----
struct OuterSide {
  const float* v;        // [T, r] by position
  const uint32_t* max;   // its largest magnitudes, one a block
  const void* x;         // [T, n] rows
  int64_t ldx;
  const float* scale;    // of the result, or nullptr
  void* out;             // [J, r, n]
  int n, vec, tiles;
};
struct OuterArgs {
  Segments seg;
  OuterSide side[2];
  int r, blocks, out_dtype;
  int tile, each;  // the blocks of `max`: `each` for every tile of so many positions
};

constexpr int kOuterThreads = 256;
constexpr int kOuterRows = 32;  // positions of a stage
constexpr int kOuterStages = 3;
constexpr int kOuterAhead = 32;  // stages whose rows are looked up at once
template <int RT>
constexpr int kOuterCols = RT <= 32 ? 256 : 128;
template <int RT>
constexpr int kOuterPerSm = RT == 16 ? 3 : RT <= 64 ? 2 : 1;  // CTAs
// 16-bit terms of v: bf16 three (24 bits), fp16 two (22 bits)
template <typename T>
constexpr int kTerms = std::is_same<T, __half>::value ? 2 : 3;

// What the sums over positions of RT ranks need.
template <typename T, int RT>
struct OuterShape {
  static constexpr int kTerm = kTerms<T>;
  static constexpr int kChunk = kOuterRows * 128;  // 64 columns or ranks of a stage
  static constexpr int kX = kOuterCols<RT> / 64 * kChunk, kV = kOuterRows * RT * 4;
  static constexpr int kPlanes = (RT * kTerm + 63) / 64 * kChunk;  // the terms of v
  // terms side by side in an accumulator, or added up in it
  static constexpr int kStacked = RT <= 64 ? kTerm : 1, kParts = kTerm / kStacked;
  static constexpr int kN = RT * kStacked;
  static constexpr int kUsed = kOuterCols<RT> / 128 * kN;  // columns of tensor memory
  // (The CTAs of kernels with clusters that fit an SM's shared memory together never want more than
  // its 512 columns, whatever their ranks: no CTA waits for columns while its cluster holds others.)
  static constexpr int kTmem = kUsed <= 64 ? 64 : kUsed <= 128 ? 128 : 256;
  // stages until an accumulator has sixteen MMAs (18 where terms are added up)
  static constexpr int kFlush = kParts == 1 ? 8 : 9 / kParts;
  static constexpr int kBytes =
      1024 + kOuterStages * (kX + kV) + 2 * kPlanes + 2 * kOuterAhead * kOuterRows * 4;
  static_assert(RT * kOuterCols<RT> * 4 <= kOuterStages * kX + 2 * kPlanes + kOuterStages * kV, "");
};

// Sums over the positions of an adapter, a tile of columns for all ranks, through tcgen05: M is
// 128 columns, K the positions, N the ranks of all terms side by side (of 128 ranks: of one term
// after the other).  Rows of x and terms of v lie as the MMAs read them, both transposed.  After
// every kFlush stages the accumulators are added, rounded, to sums in registers: MMAs cut theirs
// off where fp32 ends.  Waits for stages at 44% issue: 201 MB of x and dy at rank 16 in 51 us, 4.1
// TB/s; at ranks 64 (5120 and 5120) and 128 (2048 and 2048) 110 and 102 us at 44 and 30% issue, where
// the terms of v are made again for each tile of columns.  With mma.sync and ldmatrix the gradients
// of 8192 rows took 107 us instead of 104 (rank 16, 7168 and 5120 channels), 218 instead of 177 (64,
// 5120 and 5120) and 260 instead of 203 (128, 2048 and 2048); the split of positions has changed
// since.  Columns in twos of 128 up to 32 ranks, as tensor memory holds two CTAs' sums.
template <typename T, int RT>
__global__ void __launch_bounds__(kOuterThreads, kOuterPerSm<RT>) adapters_outer_kernel(OuterArgs a) {
  extern __shared__ unsigned char raw[];
  __shared__ uint64_t bars[kOuterStages];
  __shared__ uint32_t tmem_slot;
  using O = OuterShape<T, RT>;
  constexpr int kCols = kOuterCols<RT>, kPieces = kCols / 8, kBlocks = kCols / 128;
  constexpr int kX = O::kX, kV = O::kV, kPlanes = O::kPlanes, kTerm = kTerms<T>;
  const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;
  unsigned char* const smem = raw + (base - smem_u32(raw));
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int rank = blockIdx.x, S = gridDim.x, j = blockIdx.z, r = a.r;
  const bool second = (int)blockIdx.y >= a.side[0].tiles;
  const OuterSide& s = a.side[second];
  const int n0 = (blockIdx.y - (second ? a.side[0].tiles : 0)) * kCols;
  const uint32_t planes = base + kOuterStages * kX, vring = planes + 2 * kPlanes;
  int* rows = reinterpret_cast<int*>(smem + kOuterStages * (kX + kV) + 2 * kPlanes);
  pdl_wait();
  const int lo = a.seg.at(j), hi = max(lo, a.seg.at(j + 1));
  // this rank's positions: whole stages
  const int stages = (hi - lo + kOuterRows - 1) / kOuterRows;
  const int q0 = (int)((int64_t)stages * rank / S), q1 = (int)((int64_t)stages * (rank + 1) / S);
  float up = 1.f, down = s.scale ? s.scale[j] : 1.f;
  if constexpr (kTerm == 2) {
    uint32_t most = 0u;
    // of the adapter's own positions: what the others hold changes nothing
    const int first = (a.tile == 1 ? lo : a.seg.tiles_before(j, a.tile)) * a.each;
    const int end = min(a.blocks, first + (hi - lo + a.tile - 1) / a.tile * a.each);
    for (int i = first + tid; i < end; i += kOuterThreads) most = max(most, s.max[i]);
    const uint32_t bits = fp16_range_bits(block_max(most));
    up = __uint_as_float(bits);
    down *= inverse_pow2(bits);
  }
  // The rows of the positions, kOuterAhead stages at once, in two buffers.
  auto look_up = [&](int q) {
    int* to = rows + (q - q0) / kOuterAhead % 2 * kOuterAhead * kOuterRows;
    for (int e = tid; e < kOuterAhead * kOuterRows; e += kOuterThreads) {
      const int p = lo + q * kOuterRows + e;
      to[e] = p < hi ? a.seg.row(p) : -1;
    }
  };
  // A stage's pieces of x, and four ranks of v at once by the threads that split them (those
  // of a position without a row are zero).
  constexpr int kQuads = kOuterRows * RT / 4, kMine = (kQuads + kOuterThreads - 1) / kOuterThreads;
  const bool vvec = r % 4 == 0;
  auto load = [&](int q, int slot) {
    const int* from = rows + (q - q0) % (2 * kOuterAhead) * kOuterRows;
#pragma unroll
    for (int m = 0; m < kOuterRows * kPieces / kOuterThreads; ++m) {
      const int i = tid / kPieces + m * (kOuterThreads / kPieces), piece = tid % kPieces;
      const int row = from[i];
      stage_piece<T>(base + slot * kX + piece / 8 * O::kChunk + i * 128 +
                         (((piece % 8) ^ (i % 8)) * 16),
                     static_cast<const T*>(s.x) + (row >= 0 ? row * s.ldx : 0), n0 / 8 + piece, s.n,
                     s.vec, row >= 0);
    }
#pragma unroll
    for (int m = 0; m < kMine; ++m) {
      const int e = tid + m * kOuterThreads, i = e / (RT / 4), k = e % (RT / 4) * 4;
      if (e >= kQuads) break;
      const int p = lo + q * kOuterRows + i;
      const uint32_t to = vring + slot * kV + e * 16;
      const float* at = s.v + (int64_t)p * r + k;
      if (vvec) {
        const bool in = p < hi && k < r;
        cp_async16_or_zero(to, in ? at : s.v, in);
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const bool in = p < hi && k + c < r;
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to + 4 * c),
                       "l"(in ? at + c : s.v), "r"(in ? 4 : 0)
                       : "memory");
        }
      }
    }
  };
  auto split_v = [&](int slot, int buf) {
#pragma unroll
    for (int m = 0; m < kMine; ++m) {
      const int e = tid + m * kOuterThreads, i = e / (RT / 4), k = e % (RT / 4) * 4;
      if (e >= kQuads) break;
      float f[4];
      asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3])
                   : "r"(vring + slot * kV + e * 16)
                   : "memory");
#pragma unroll
      for (int c = 0; c < 4; ++c) f[c] *= up;
#pragma unroll
      for (int t = 0; t < kTerm; ++t) {
        const uint32_t w0 = pack2<T>(f[0], f[1]), w1 = pack2<T>(f[2], f[3]);
        const int n = t * RT + k;
        const uint32_t at = planes + buf * kPlanes + n / 64 * O::kChunk + i * 128 +
                            (((n % 64 / 8) ^ (i % 8)) * 16) + n % 8 * 2;
        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at), "r"(w0), "r"(w1) : "memory");
        const float2 g0 = unpack2<T>(w0), g1 = unpack2<T>(w1);
        f[0] = left_of(f[0], g0.x);
        f[1] = left_of(f[1], g0.y);
        f[2] = left_of(f[2], g1.x);
        f[3] = left_of(f[3], g1.y);
      }
    }
  };
  look_up(q0);
  if (tid == 0) {
#pragma unroll
    for (int q = 0; q < kOuterStages; ++q) mbar_init(smem_u32(&bars[q]), 1);
    fence_barrier_init();
  }
  __syncwarp();
  if (warp == 0) tmem_alloc(smem_u32(&tmem_slot), O::kTmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();  // (every CTA has its tensor memory before another kernel's CTAs take theirs)
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&tmem_slot);
#pragma unroll
  for (int i = 0; i < kOuterStages - 1; ++i) {
    if (q0 + i < q1) load(q0 + i, i);
    cp_async_commit();
  }
  const uint32_t idesc = (std::is_same<T, __half>::value ? idesc_f16_f32(128, O::kN)
                                                         : idesc_bf16_f32(128, O::kN)) |
                         (1u << 15) | (1u << 16);  // columns, and ranks, side by side
  // a thread has a column, and half of the ranks where the tile is 128 columns
  constexpr int kSums = RT * kBlocks / 2;
  const int block = kBlocks == 2 ? warp / 4 : 0, first = kBlocks == 2 ? 0 : warp / 4 * kSums;
  float sum[kSums] = {};
  bool ok = true;
  for (int q = q0; q < q1; ++q) {
    const int n = q - q0, buf = n & 1, slot = n % kOuterStages;
    cp_async_wait<kOuterStages - 2>();
    split_v(slot, buf);  // what this thread copied
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    if (tid == 0) {
      tc_fence_after();
#pragma unroll
      for (int m = 0; m < kBlocks; ++m)
#pragma unroll
        for (int t = 0; t < O::kParts; ++t)
#pragma unroll
          for (int k = 0; k < kOuterRows / 16; ++k)
            tc_mma_bf16(tmem + m * O::kN,
                        sdesc_rows(base + slot * kX + m * 2 * O::kChunk + k * 2048, O::kChunk),
                        sdesc_rows(planes + buf * kPlanes + t * (O::kN / 64 * O::kChunk) + k * 2048,
                                   O::kChunk),
                        idesc, n % O::kFlush > 0 || t > 0 || k > 0);
      tc_commit(smem_u32(&bars[slot]));
    }
    __syncwarp();
    // the stage before is free when its MMAs are done
    if (n > 0) ok = warp_wait(smem_u32(&bars[(n - 1) % kOuterStages]),
                              (n - 1) / kOuterStages & 1) && ok;
    const int ahead = q + kOuterStages - 1;
    if (ahead < q1) load(ahead, (ahead - q0) % kOuterStages);
    cp_async_commit();
    if (n % kOuterAhead == 0 && q + kOuterAhead < q1) look_up(q + kOuterAhead);
    if (n % O::kFlush == O::kFlush - 1 || q == q1 - 1) {
      ok = warp_wait(smem_u32(&bars[slot]), n / kOuterStages & 1) && ok;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < kSums; c += 16) {
        uint32_t d[kTerm][16];
#pragma unroll
        for (int t = 0; t < O::kStacked; ++t)
          tmem_ld16(tmem + ((uint32_t)(warp % 4 * 32) << 16) + block * O::kN + t * RT + first + c, d[t]);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float f = __uint_as_float(d[0][i]);
#pragma unroll
          for (int t = 1; t < O::kStacked; ++t) f += __uint_as_float(d[t][i]);
          sum[c + i] += f;
        }
      }
    }
  }
  tc_fence_before();
  cp_async_wait<0>();
  __syncthreads();
  // parts [rank][column], added in the order of the cluster's ranks
  float* red = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int i = 0; i < kSums; ++i)
    red[(first + i) * kCols + block * 128 + warp % 4 * 32 + lane] = ok ? sum[i] : NAN;
  cluster_sync_all();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, O::kTmem);
  }
  for (int e = rank * kOuterThreads + tid; e < r * kCols; e += S * kOuterThreads) {
    const int i = e / kCols, n = n0 + e % kCols;
    if (n >= s.n) continue;
    float f = 0.f;
    for (int q = 0; q < S; ++q) f += ld_cluster_f32(mapa_shared(base + e * 4, q));
    f *= down;
    const int64_t at = ((int64_t)j * r + i) * s.n + n;
    if (a.out_dtype == MOE_DT_FP32)
      static_cast<float*>(s.out)[at] = f;
    else
      static_cast<T*>(s.out)[at] = from_f<T>(f);
  }
  cluster_sync_all();
}

// ------------------------------------------------------------------ launch --
template <int RT>
constexpr int shrink_smem() {
  // (on the tensor cores from a 1024-byte boundary on)
  return kShrinkStages * (kShrinkRows<RT> + RT) * 128 + (RT <= 64 ? 0 : 1024);
}

// CTAs of the shrink that an SM's shared memory holds, as the split over K counts them.  Rank 128,
// 5120 to 5120 channels, where one fits: 8192 rows 130 us, counted as two 138; 4096 rows 81 and 101.
constexpr int shrink_per_sm(int r) { return r <= 32 ? 4 : r <= 64 ? 2 : 1; }
static_assert(shrink_per_sm(16) * (shrink_smem<16>() + 1024) <= 228 * 1024 &&
                  shrink_per_sm(32) * (shrink_smem<32>() + 1024) <= 228 * 1024 &&
                  shrink_per_sm(64) * (shrink_smem<64>() + 1024) <= 228 * 1024 &&
                  shrink_per_sm(128) * (shrink_smem<128>() + 1024) <= 228 * 1024,
              "CTAs of one round");

// The most CTAs of a power of two, up to eight, that share `units` of work while there
// are at most `most` CTAs in all and each has at least `least` units.
int adapters_split(int64_t clusters, int64_t units, int64_t most, int64_t least) {
  int s = 1;
  while (s < kMaxCluster && clusters * 2 * s <= most && units >= 2 * s * least) s *= 2;
  return s;
}

// One position a cluster, or tiles of positions.  By rows every row reads its adapter again
// (from L2): cheap while that is little, or where adapters have about a row each; the offsets that
// say how many have rows lie on the device, so many loaded adapters count as that while T is small
// beside the SMs.  us by rows and in tiles: rank 16, 5120 to 5120 channels, 64 rows 9.1 and 15.6, 128
// (21 M products) 15.6 and 16.1, 160 21.5 and 16.2; 1000 to 1000, 300 rows 8.5 and 10.0, 1000 rows 25
// and 10.7; rank 32, 2048 to 2048, 64 rows (8.4 M) 10.6 and 10.2, 128 19 and 11; rank 64, 40 rows 16.5
// and 12.5; 64 rows of 64 adapters, rank 64, 2048 to 2048 19 and 29, of 48, rank 16, 7168 to 2048 9.3
// and 20.  1024 loaded adapters, rows of all of them, and of one (captured in a graph): rank 16, 5120
// to 5120, 512 rows 81 and 199, 71 and 134, 2048 rows 253 and 353, 237 and 159; rank 64, 2048 to 2048,
// 256 rows 79 and 118, 67 and 73, 512 rows 140 and 207, 120 and 89, 2048 rows 470 and 407, 433 and
// 128; rank 128, 5120 to 5120, 512 rows 335 and 724, 249 and 245, 2048 rows 1042 and 1515, 945 and 335.
bool adapters_by_rows(const AdapterArgs& a, int num_sms) {
  const int64_t T = a.seg.T;
  return (T <= 2 * a.seg.J && T <= (a.r <= 16 ? 8 : 3) * num_sms) ||
         (T <= 2 * num_sms && T * a.r * (a.K + a.N) <= (a.r <= 16 ? 20 << 20 : 8 << 20));
}

int row_cluster(const AdapterArgs& a) {
  // slices of at least 256 channels
  return adapters_split(1, std::max(a.K, a.N), kMaxCluster, 256);
}
// Warps of a CTA: for all ranks at once, where clusters of that many surely find room together (an
// SM holds sixteen warps; GPCs are not filled evenly).  One row, 5120 to 5120 channels, rank 64: 16.1
// us with four, 9.0 with sixteen; 128: 27.8 and 13.5; but 64 rows of 64 adapters, 2048 to 2048, rank
// 64: 19 and 36.
int row_warps(const AdapterArgs& a, int cluster, int num_sms) {
  int warps = a.r <= 16 ? 4 : a.r <= 32 ? 8 : 16;
  while (warps > 4 && (int64_t)a.seg.T * cluster * warps * 2 > 16LL * num_sms) warps /= 2;
  return warps;
}
// Tiles of `rows` positions that may have any: see Segments::tile.
int adapter_tiles(const AdapterArgs& a, int rows) {
  return a.seg.T / rows + std::min(a.seg.J + 1, a.seg.T) + (a.seg.T % rows ? 1 : 0);
}
int shrink_cluster(const AdapterArgs& a, int num_sms) {
  const int rows = shrink_rows(a.r);
  return adapters_split((a.seg.T + rows - 1) / rows, (a.K + 63) / 64,
                        (int64_t)shrink_per_sm(a.r) * num_sms, 4);
}

template <typename T, int RT>
void launch_tiles(const Launch& L, const AdapterArgs& a, int rt_slot) {
  const int type = std::is_same<T, __half>::value ? 1 : 0;
  const int S = shrink_cluster(a, L.num_sms);
  auto shrink = [&](auto kernel) {
    set_smem_attr_once(reinterpret_cast<const void*>(kernel), shrink_smem<RT>(),
                       kAttrAdapters + 8 * type + rt_slot);
    launch_begin(L, MOE_K_ADAPTERS);
    launch_kernel_cluster(kernel, dim3(S, adapter_tiles(a, kShrinkRows<RT>)), dim3(S),
                          dim3(2 * kShrinkRows<RT>), shrink_smem<RT>(), L.stream, a);
    launch_end(L, MOE_K_ADAPTERS);
  };
  if constexpr (RT <= 64)
    shrink(adapters_shrink_kernel<T, RT>);
  else
    shrink(adapters_shrink_tc_kernel<T, RT>);
  if (!a.y) return;
  // ranges of whole tiles of columns, for one round of CTAs: a CTA has about as long to start
  // (tile, rows, v) as for several tiles of columns (at most 4 or 6 of them a CTA, 640 or 448 CTAs
  // where 256 do: 84 us instead of 78 at 8192 rows and rank 64; adapters whose rows are fewer than
  // a tile's have one each)
  const int blocks = std::max((a.seg.T + kExpandRows - 1) / kExpandRows +
                                  std::min(a.seg.J, a.seg.T) / 2, std::min(a.seg.J, a.seg.T));
  const int tiles = (a.N + kExpandTile - 1) / kExpandTile;
  const int ranges = std::max(1, std::min(tiles, kExpandPerSm<RT> * L.num_sms / blocks));
  const int per = (tiles + ranges - 1) / ranges;
  constexpr int kSmem = 1024 + 2 * ((RT + 63) / 64 * kExpandRows * 128 + RT * kExpandTile * 2);
  auto expand = [&](auto kernel, int slot) {
    set_smem_attr_once(reinterpret_cast<const void*>(kernel), kSmem, kAttrAdapters + slot);
    launch_begin(L, MOE_K_ADAPTERS);
    launch_kernel(kernel, dim3((tiles + per - 1) / per, adapter_tiles(a, kExpandRows)),
                  dim3(kExpandThreads), kSmem, L.stream, a, per * kExpandTile);
    launch_end(L, MOE_K_ADAPTERS);
  };
  if constexpr (RT <= 32) {
    if (a.base) {
      expand(adapters_expand_kernel<T, RT, true>, 24 + 2 * type + rt_slot);
      return;
    }
  }
  expand(adapters_expand_kernel<T, RT, false>, 8 * type + 4 + rt_slot);
}
template <typename T, int RT>
void launch_outer(const Launch& L, OuterArgs a, int rt_slot) {
  const int type = std::is_same<T, __half>::value ? 1 : 0;
  int tiles = 0;
  for (OuterSide& s : a.side) {
    s.tiles = (s.n + kOuterCols<RT> - 1) / kOuterCols<RT>;
    tiles += s.tiles;
  }
  // the split of an adapter's positions with the least time by a count of stages: rounds of
  // CTAs, each of its stages and about eight more to start and to add the parts (with four 8192 rows,
  // 5120 to 5120, rank 64 177 us instead of 164)
  const int64_t clusters = (int64_t)tiles * a.seg.J, slots = (int64_t)kOuterPerSm<RT> * L.num_sms;
  const int64_t stages = std::max(1, a.seg.T / a.seg.J / kOuterRows);
  int S = 1;
  int64_t least = INT64_MAX;
  for (int q = 1; q <= kMaxCluster; ++q) {
    const int64_t cost = (clusters * q + slots - 1) / slots * ((stages + q - 1) / q + 8);
    if (cost < least) {
      least = cost;
      S = q;
    }
  }
  set_smem_attr_once(reinterpret_cast<const void*>(adapters_outer_kernel<T, RT>),
                     OuterShape<T, RT>::kBytes, kAttrAdapters + 16 + 4 * type + rt_slot);
  launch_begin(L, MOE_K_ADAPTERS_GRAD);
  launch_kernel_cluster(adapters_outer_kernel<T, RT>, dim3(S, tiles, a.seg.J), dim3(S),
                        dim3(kOuterThreads), OuterShape<T, RT>::kBytes, L.stream, a);
  launch_end(L, MOE_K_ADAPTERS_GRAD);
}

// Shrink and expand, then (outer not nullptr) the sums over positions.
template <typename T>
void launch_adapters(const Launch& L, const AdapterArgs& a, OuterArgs* outer) {
  const int slot = a.r <= 16 ? 0 : a.r <= 32 ? 1 : a.r <= 64 ? 2 : 3;
  if (a.seg.T == 0) {
  } else if (adapters_by_rows(a, L.num_sms)) {
    const int C = row_cluster(a);
    launch_begin(L, MOE_K_ADAPTERS);
    auto rows = [&](auto kernel, int warps) {
      launch_kernel_cluster(kernel, dim3(C, a.seg.T), dim3(C), dim3(32 * warps), 0, L.stream, a);
    };
    switch (row_warps(a, C, L.num_sms)) {
      case 4: rows(adapters_row_kernel<T, 4>, 4); break;
      case 8: rows(adapters_row_kernel<T, 8>, 8); break;
      default: rows(adapters_row_kernel<T, 16>, 16); break;
    }
    launch_end(L, MOE_K_ADAPTERS);
    if (outer) {
      outer->tile = 1;
      outer->each = C;
      outer->blocks = C * a.seg.T;
    }
  } else {
    switch (slot) {
      case 0: launch_tiles<T, 16>(L, a, 0); break;
      case 1: launch_tiles<T, 32>(L, a, 1); break;
      case 2: launch_tiles<T, 64>(L, a, 2); break;
      default: launch_tiles<T, 128>(L, a, 3); break;
    }
    if (outer) {
      outer->tile = shrink_rows(a.r);
      outer->each = shrink_cluster(a, L.num_sms);
      outer->blocks = outer->each * adapter_tiles(a, outer->tile);
    }
  }
  if (!outer) return;
  switch (slot) {
    case 0: launch_outer<T, 16>(L, *outer, 0); break;
    case 1: launch_outer<T, 32>(L, *outer, 1); break;
    case 2: launch_outer<T, 64>(L, *outer, 2); break;
    default: launch_outer<T, 128>(L, *outer, 3); break;
  }
}

struct AdapterLayout {
  size_t v, max_v, max_other, total;
};
AdapterLayout adapters_layout(int64_t T, int64_t r) {
  auto up = [](int64_t n) { return ((size_t)n + 255) & ~(size_t)255; };
  // largest magnitudes: a word for each CTA of a position's cluster or of a tile's, of which there
  // are at most T / 64 + T + 1 (adapter_tiles)
  const int64_t words = T > 0 ? kMaxCluster * (T + T / 64 + 2) : 0;
  AdapterLayout l;
  l.v = 0;
  l.max_v = up(T * r * 4);
  l.max_other = l.max_v + up(words * 4);
  l.total = l.max_other + up(words * 4);
  return l;
}

moe_status check_adapters(int32_t T, int32_t J, int32_t r, int32_t K, int32_t N, int32_t dtype) {
  if (T < 0 || J < 1 || r < 1 || K < 1 || N < 1) return MOE_ERR_INVALID_ARG;
  if (dtype != MOE_DT_BF16 && dtype != MOE_DT_FP16) return MOE_ERR_INVALID_ARG;
  if (r > kMaxRank || J > kMaxAdapters || T > (1 << 21) || K > (1 << 21) || N > (1 << 21))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_adapters_workspace_size(int32_t T, int32_t r, int32_t K,
                                                  int32_t N, size_t* bytes) {
  const moe_status s = check_adapters(T, 1, r, K, N, MOE_DT_BF16);
  if (s != MOE_OK) return s;
  if (!bytes) return MOE_ERR_INVALID_ARG;
  *bytes = adapters_layout(T, r).total;
  return MOE_OK;
}

extern "C" moe_status moe_adapters(int32_t T, int32_t n_adapters, int32_t r, int32_t K, int32_t N,
                                   int32_t dtype, const void* x, int64_t ldx, const void* a,
                                   const void* b, const float* scale, const int32_t* offsets,
                                   const int32_t* order, const void* base, int64_t ldb, void* y,
                                   int64_t ldy, float* v, void* ws, size_t ws_bytes,
                                   moe_stream_t stream) {
  const moe_status cs = check_adapters(T, n_adapters, r, K, N, dtype);
  if (cs != MOE_OK) return cs;
  if (ldx < K || (base && ldb < N) || ldy < N) return MOE_ERR_INVALID_ARG;
  if (base && base == y && ldb != ldy) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!x || !a || !b || !offsets || !y || !ws) return MOE_ERR_INVALID_ARG;
  if (misaligned16(x, a, b, scale, offsets, order, base, y, v) ||
      (reinterpret_cast<uintptr_t>(ws) & 255u))
    return MOE_ERR_ALIGNMENT;
  const AdapterLayout l = adapters_layout(T, r);
  if (ws_bytes < l.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (y == x) return MOE_ERR_INVALID_ARG;
  Launch L;
  const moe_status s = open_launch(stream, &L);
  if (s != MOE_OK) return s;
  AdapterArgs g{};
  g.seg = {offsets, order, T, n_adapters};
  g.x = x;
  g.ldx = ldx;
  g.m1 = a;
  g.v = v ? v : reinterpret_cast<float*>(static_cast<char*>(ws) + l.v);
  g.m2 = b;
  g.scale2 = scale;
  g.base = base;
  g.ldb = ldb;
  g.y = y;
  g.ldy = ldy;
  g.r = r;
  g.K = K;
  g.N = N;
  g.xvec = K % 8 == 0 && ldx % 8 == 0;
  g.m1vec = K % 8 == 0;
  g.m2vec = N % 8 == 0;
  g.yvec = N % 8 == 0 && ldy % 8 == 0 && (!base || ldb % 8 == 0);
  if (dtype == MOE_DT_BF16)
    launch_adapters<__nv_bfloat16>(L, g, nullptr);
  else
    launch_adapters<__half>(L, g, nullptr);
  return launch_status_take();
}

extern "C" moe_status moe_adapters_backward(
    int32_t T, int32_t n_adapters, int32_t r, int32_t K, int32_t N, int32_t dtype, const void* dy,
    int64_t lddy, const void* x, int64_t ldx, const float* v, const void* a, const void* b,
    const float* scale, const int32_t* offsets, const int32_t* order, void* dx, int64_t lddx,
    int32_t grad_dtype, void* da, void* db, void* ws, size_t ws_bytes, moe_stream_t stream) {
  const moe_status cs = check_adapters(T, n_adapters, r, K, N, dtype);
  if (cs != MOE_OK) return cs;
  if (lddy < N || ldx < K || (dx && lddx < K)) return MOE_ERR_INVALID_ARG;
  if ((da != nullptr) != (db != nullptr) || (!dx && !da)) return MOE_ERR_INVALID_ARG;
  if (da && grad_dtype != MOE_DT_FP32 && grad_dtype != dtype) return MOE_ERR_INVALID_ARG;
  if (!offsets || !a || !b) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!dy || !ws || (da && (!x || !v)))) return MOE_ERR_INVALID_ARG;
  if (misaligned16(dy, x, v, a, b, scale, offsets, order, dx, da, db) ||
      (reinterpret_cast<uintptr_t>(ws) & 255u))
    return MOE_ERR_ALIGNMENT;
  const AdapterLayout l = adapters_layout(T, r);
  if (ws_bytes < l.total) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if (T == 0 && !da) return MOE_OK;
  if (T > 0 && dx && (dx == dy || dx == x)) return MOE_ERR_INVALID_ARG;
  Launch L;
  const moe_status s = open_launch(stream, &L);
  if (s != MOE_OK) return s;
  char* at = static_cast<char*>(ws);
  AdapterArgs g{};
  g.seg = {offsets, order, T, n_adapters};
  g.x = dy;
  g.ldx = lddy;
  g.m1 = b;
  g.scale1 = scale;
  g.v = reinterpret_cast<float*>(at + l.v);
  g.m2 = a;
  g.y = dx;
  g.ldy = lddx;
  g.r = r;
  g.K = N;
  g.N = K;
  g.xvec = N % 8 == 0 && lddy % 8 == 0;
  g.m1vec = N % 8 == 0;
  g.m2vec = K % 8 == 0;
  g.yvec = K % 8 == 0 && lddx % 8 == 0;
  OuterArgs o{};
  if (da) {
    g.other = v;
    g.max_v = reinterpret_cast<uint32_t*>(at + l.max_v);
    g.max_other = reinterpret_cast<uint32_t*>(at + l.max_other);
    o.seg = g.seg;
    o.side[0] = {g.v, g.max_v, x, ldx, nullptr, da, K, K % 8 == 0 && ldx % 8 == 0, 0};
    o.side[1] = {v, g.max_other, dy, lddy, scale, db, N, g.xvec, 0};
    o.r = r;
    o.out_dtype = grad_dtype;
  }
  if (dtype == MOE_DT_BF16)
    launch_adapters<__nv_bfloat16>(L, g, da ? &o : nullptr);
  else
    launch_adapters<__half>(L, g, da ? &o : nullptr);
  return launch_status_take();
}
