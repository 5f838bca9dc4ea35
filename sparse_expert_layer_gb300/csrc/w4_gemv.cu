// Matrix-vector products with 4-bit weights and group scales, expert by expert.
//
//   out[r, n] = sum over groups g of s[n, g] * sum over k in g of (q[n, k] - z[n, g]) * x[r, k]
//
// for the rows r of each expert; with a second matrix, silu(first) * second.
//
// A weight is half a byte, so at the memory rate each SM has to take in about
// 47 weights a cycle; one multiply-add a weight and row on CUDA cores would cost
// more than that at two rows, so the products run as warp-level MMAs with the
// weights as the 16-row operand and up to eight token rows as the other.  The
// integers q - z are exact in bf16 and fp16, their products with x are exact in
// the MMA's fp32 accumulators, and a group's sum is multiplied by its scale in
// fp32, so nothing is rounded but the fp32 sums and the output.
//
// A CTA takes 128 weight rows (128 channels, or 64 of both matrices) and a range
// of K; its eight warps are four row tiles of 32 times two halves of each
// 512-wide panel.  Every warp streams its own weights through a ring of
// cp.async stages, so no barrier stands between weights and MMAs; only the
// panels of x and scales are shared.  With few row tiles a cluster of CTAs
// splits K and adds the parts through distributed shared memory in rank order.
#include <math.h>

#include <algorithm>

#include "rows.cuh"

namespace moe {

namespace {

constexpr int kW4MaxExperts = 4096;
constexpr int kW4Warps = 8;
constexpr int kW4Threads = 32 * kW4Warps;
constexpr int kW4Rows = 128;               // weight rows of a CTA
constexpr int kW4Panel = 512;              // K of a panel of x and scales
constexpr int kW4Stage = 128;              // K of a ring stage
constexpr int kW4Stages = 4;
constexpr int kW4RowBytes = kW4Stage / 2 + 16;  // padded: ldmatrix rows fall in distinct banks
constexpr int kW4StageBytes = 32 * kW4RowBytes;
constexpr int kW4RedStride = kW4Rows + 4;
constexpr int kW4MaxSplit = 8;

struct W4Args {
  const int32_t* offsets;  // [E + 1], nullptr: one expert with all R rows
  const void* x;
  const float* x_scale;
  const uint8_t* w[2];
  const void* s[2];
  const uint8_t* z[2];
  void* out;
  int E, N, K, R, groups, group;
  int channels;   // channels of a CTA: 128, or 64 with a second matrix
  int up;
  int scale_dtype, out_dtype;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool real) {
  const int n = real ? 16 : 0;  // 0: the 16 bytes become zeros, src is not read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// The 16-bit type of the MMA: bf16, or fp16.
struct MmaBf16 {
  static constexpr uint32_t kMagic = 0x43004300u;  // 128: a nibble below makes 128 + q
  static __device__ __forceinline__ uint32_t sub(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                             uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};
struct MmaFp16 {
  static constexpr uint32_t kMagic = 0x64006400u;  // 1024
  static __device__ __forceinline__ uint32_t sub(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                             uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};

// The x types: bytes of a channel, the MMA type, and a thread's eight channels
// k0 .. k7 of one row as the four words (k0,k4) (k1,k5) (k2,k6) (k3,k7), the
// order in which the nibbles of a weight word pair up.
struct XBf16 {
  using Mma = MmaBf16;
  static constexpr int kBytes = 2;
  static constexpr int kStride = kW4Panel * 2 + 64;  // rows 64 bytes apart modulo the banks
  static __device__ __forceinline__ void pairs(const unsigned char* p, uint32_t (&b)[4]) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    b[0] = __byte_perm(v.x, v.z, 0x5410);
    b[1] = __byte_perm(v.x, v.z, 0x7632);
    b[2] = __byte_perm(v.y, v.w, 0x5410);
    b[3] = __byte_perm(v.y, v.w, 0x7632);
  }
};
struct XFp16 : XBf16 {
  using Mma = MmaFp16;
};
// int8 codes: fp16 holds them exactly, 1024 + (code + 128) below the mantissa
// less 1152; a group's sum of at most 128 products stays below 2^24, exact.
struct XInt8 {
  using Mma = MmaFp16;
  static constexpr int kBytes = 1;
  static constexpr int kStride = kW4Panel + 32;
  static __device__ __forceinline__ void pairs(const unsigned char* p, uint32_t (&b)[4]) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    const uint32_t lo = v.x ^ 0x80808080u, hi = v.y ^ 0x80808080u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // bytes (k_i, k_{i+4}) into the low bytes of two halves under 0x64
      const uint32_t both = __byte_perm(lo, hi, i | ((4 + i) << 4));
      b[i] = MmaFp16::sub(__byte_perm(both, 0x64646464u, 0x4140), 0x64806480u);
    }
  }
};

// A weight word holds channels k0 .. k7, a nibble each, k0 lowest: pair i is
// (q(k_i) - z, q(k_{i+4}) - z) in 16 bits each, exact.
template <typename M>
__device__ __forceinline__ uint32_t dequant_pair(uint32_t w, int i, uint32_t zero) {
  const uint32_t v = ((w >> (4 * i)) & 0x000f000fu) | M::kMagic;
  return M::sub(v, zero);
}

__device__ __forceinline__ float load_scale(const void* s, int dtype, int64_t i) {
  if (dtype == MOE_DT_BF16) return to_f(static_cast<const __nv_bfloat16*>(s)[i]);
  if (dtype == MOE_DT_FP16) return to_f(static_cast<const __half*>(s)[i]);
  return static_cast<const float*>(s)[i];
}

__host__ __device__ constexpr int panel_groups(int group, int K) {
  return group == K || group >= kW4Panel ? 1 : kW4Panel / group;
}

template <typename X, int NB>
struct W4Smem {
  static constexpr int kRing = kW4Warps * kW4Stages * kW4StageBytes;
  static constexpr int kX = NB * 8 * X::kStride;
  static constexpr int kRed = NB * 8 * kW4RedStride * 4;
  static int bytes(int pgroups, bool zeros) {
    return kRing + 2 * kX + 2 * pgroups * kW4Rows * (zeros ? 8 : 4) + kRed;
  }
};

// NB: blocks of eight token rows per pass over the weights.  GS: 32-wide K steps
// after which a group's sum is scaled (group 32: 1, 64: 2, else 4).
template <typename X, int NB, int GS, bool ZEROS>
__global__ void __launch_bounds__(kW4Threads, 2) w4_gemv_kernel(W4Args a) {
  pdl_enter();
  using M = typename X::Mma;
  using S = W4Smem<X, NB>;
  extern __shared__ __align__(128) unsigned char smem[];
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int nw = warp % 4, kw = warp / 4;
  const int g = lane / 4, c = lane % 4;
  const int e = blockIdx.z, split = gridDim.x, rank = blockIdx.x;
  int row0 = 0, row1 = a.R;
  if (a.offsets) {  // offsets are data: stay inside the R rows whatever they hold
    row0 = min(max(a.offsets[e], 0), a.R);
    row1 = min(max(a.offsets[e + 1], row0), a.R);
  }
  if (row0 == row1) return;  // the whole cluster

  const int pg = panel_groups(a.group, a.K);
  unsigned char* xs = smem + S::kRing;
  float* scales = reinterpret_cast<float*>(xs + 2 * S::kX);          // [2][pg][128]
  uint32_t* zeros = reinterpret_cast<uint32_t*>(scales + 2 * pg * kW4Rows);
  float* red = reinterpret_cast<float*>(zeros + (ZEROS ? 2 * pg * kW4Rows : 0));
  const uint32_t ring = smem_u32(smem) + warp * kW4Stages * kW4StageBytes;

  // weight row i (0 .. 127) of the CTA: warp tile i / 32; with a second matrix
  // rows 0-15 of a tile are the first's, 16-31 the second's, of 16 channels
  const int n0 = blockIdx.y * a.channels;
  auto row_channel = [&](int i) {
    return a.up ? n0 + (i / 32) * 16 + i % 16 : n0 + i;
  };
  auto row_matrix = [&](int i) { return a.up ? (i / 16) % 2 : 0; };

  const int panels = (a.K + kW4Panel - 1) / kW4Panel;
  const int per = (panels + split - 1) / split;
  const int p0 = min(panels, rank * per), p1 = min(panels, p0 + per);

  // this lane's four weight rows of every stage (rows i * 8 + lane / 4), 16-byte
  // piece lane % 4
  const uint8_t* wrow[4];
  bool wreal[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = nw * 32 + i * 8 + lane / 4, n = row_channel(r);
    wreal[i] = n < a.N;
    wrow[i] = a.w[row_matrix(r)] + ((int64_t)e * a.N + (wreal[i] ? n : 0)) * (a.K / 2);
  }
  // stage q of this warp covers K from p0's panel on: two stages a panel
  auto load_stage = [&](int q) {
    const int k = (p0 + q / 2) * kW4Panel + kw * (kW4Panel / 2) + (q % 2) * kW4Stage +
                  (lane % 4) * 32;
    const bool in = q < 2 * (p1 - p0) && k < a.K;
    const uint32_t dst = ring + (q % kW4Stages) * kW4StageBytes + (lane % 4) * 16;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      cp_async16(dst + (i * 8 + lane / 4) * kW4RowBytes, wrow[i] + (in ? k / 2 : 0),
                 in && wreal[i]);
    cp_async_commit();
  };

  // x: 16-byte pieces of a panel, a thread takes every 256th; scales: one of
  // the CTA's rows and every second group a thread
  constexpr int kPieces = kW4Panel * X::kBytes / 16;  // of a row
  constexpr int kXPer = NB * 8 * kPieces / kW4Threads;
  const unsigned char* xg = static_cast<const unsigned char*>(a.x);
  const int srow = tid % kW4Rows, sn = row_channel(srow);
  const bool sreal = sn < a.N;
  const int64_t sbase = ((int64_t)e * a.N + (sreal ? sn : 0)) * a.groups;
  const void* sptr = a.s[row_matrix(srow)];
  const uint8_t* zptr = a.z[row_matrix(srow)];

  for (int chunk = row0; chunk < row1; chunk += NB * 8) {
    const int m = min(NB * 8, row1 - chunk);
    uint4 xr[kXPer];
    auto fetch_x = [&](int p) {
#pragma unroll
      for (int i = 0; i < kXPer; ++i) {
        const int u = tid + i * kW4Threads, tok = u / kPieces;
        const int k = p * kW4Panel + (u % kPieces) * (16 / X::kBytes);
        xr[i] = make_uint4(0u, 0u, 0u, 0u);
        if (tok < m && k < a.K)
          xr[i] = *reinterpret_cast<const uint4*>(xg + ((int64_t)(chunk + tok) * a.K + k) *
                                                           X::kBytes);
      }
    };
    auto put_panel = [&](int p) {
      unsigned char* xb = xs + (p & 1) * S::kX;
#pragma unroll
      for (int i = 0; i < kXPer; ++i) {
        const int u = tid + i * kW4Threads;
        *reinterpret_cast<uint4*>(xb + (u / kPieces) * X::kStride + (u % kPieces) * 16) = xr[i];
      }
      for (int j = tid / kW4Rows; j < pg; j += kW4Threads / kW4Rows) {
        const int grp = (p * kW4Panel) / a.group + j;
        const bool in = sreal && grp < a.groups;
        scales[((p & 1) * pg + j) * kW4Rows + srow] =
            in ? load_scale(sptr, a.scale_dtype, sbase + grp) : 0.f;
        if constexpr (ZEROS)
          zeros[((p & 1) * pg + j) * kW4Rows + srow] =
              M::kMagic + (in ? (zptr[sbase + grp] & 31u) * 0x00010001u : 0u);
      }
    };

#pragma unroll
    for (int q = 0; q < kW4Stages - 1; ++q) load_stage(q);
    float acc[2][NB][4] = {};
    if (p0 < p1) {
      fetch_x(p0);
      put_panel(p0);
    }
    __syncthreads();
    for (int p = p0; p < p1; ++p) {
      if (p + 1 < p1) fetch_x(p + 1);
      const unsigned char* xb = xs + (p & 1) * S::kX + g * X::kStride;
      const float* sb = scales + (p & 1) * pg * kW4Rows + nw * 32 + g;
      const uint32_t* zb = zeros + (p & 1) * pg * kW4Rows + nw * 32 + g;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int q = 2 * (p - p0) + h;
        cp_async_wait<kW4Stages - 2>();
        __syncwarp();
        load_stage(q + kW4Stages - 1);
        const uint32_t st = ring + (q % kW4Stages) * kW4StageBytes + lane * kW4RowBytes;
        const int kp = kw * (kW4Panel / 2) + h * kW4Stage;  // K inside the panel
#pragma unroll
        for (int s0 = 0; s0 < 4; s0 += GS) {
          const int grp = pg == 1 ? 0 : (kp + s0 * 32) / a.group;
          uint32_t zc[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            zc[i] = ZEROS ? zb[grp * kW4Rows + i * 8] : M::kMagic + 0x00080008u;
          float part[2][NB][4] = {};
#pragma unroll
          for (int s = s0; s < s0 + GS; ++s) {
            uint32_t wv[4];  // first tile rows g, g + 8; second tile rows g, g + 8
            ldmatrix_x4(st + s * 16, wv);
            uint32_t af[2][2][4];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                af[t][i][0] = dequant_pair<M>(wv[2 * t], 2 * i, zc[2 * t]);
                af[t][i][1] = dequant_pair<M>(wv[2 * t + 1], 2 * i, zc[2 * t + 1]);
                af[t][i][2] = dequant_pair<M>(wv[2 * t], 2 * i + 1, zc[2 * t]);
                af[t][i][3] = dequant_pair<M>(wv[2 * t + 1], 2 * i + 1, zc[2 * t + 1]);
              }
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              uint32_t bf[4];
              X::pairs(xb + b * 8 * X::kStride + (kp + s * 32 + c * 8) * X::kBytes, bf);
#pragma unroll
              for (int t = 0; t < 2; ++t) {
                M::mma(part[t][b], af[t][0], bf[0], bf[1]);
                M::mma(part[t][b], af[t][1], bf[2], bf[3]);
              }
            }
          }
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const float s_lo = sb[grp * kW4Rows + t * 16], s_hi = sb[grp * kW4Rows + t * 16 + 8];
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              acc[t][b][0] = fmaf(s_lo, part[t][b][0], acc[t][b][0]);
              acc[t][b][1] = fmaf(s_lo, part[t][b][1], acc[t][b][1]);
              acc[t][b][2] = fmaf(s_hi, part[t][b][2], acc[t][b][2]);
              acc[t][b][3] = fmaf(s_hi, part[t][b][3], acc[t][b][3]);
            }
          }
        }
      }
      if (p + 1 < p1) put_panel(p + 1);
      __syncthreads();
    }
    cp_async_wait<0>();

    // add the two K halves, then the cluster's parts, in a fixed order
    auto red_at = [&](int t, int b, int j) -> float& {
      const int tok = b * 8 + 2 * c + (j & 1), r = nw * 32 + t * 16 + g + (j >> 1) * 8;
      return red[tok * kW4RedStride + r];
    };
    if (kw == 1) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int j = 0; j < 4; ++j) red_at(t, b, j) = acc[t][b][j];
    }
    __syncthreads();
    if (kw == 0) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int j = 0; j < 4; ++j) red_at(t, b, j) += acc[t][b][j];
    }
    if (split > 1)
      cluster_sync_all();
    else
      __syncthreads();
    const uint32_t red_sh = smem_u32(red);
    auto total = [&](int tok, int r) {
      if (split == 1) return red[tok * kW4RedStride + r];
      float v = 0.f;
      for (int q = 0; q < split; ++q)
        v += ld_cluster_f32(mapa_shared(red_sh + (tok * kW4RedStride + r) * 4, q));
      return v;
    };
    for (int i = tid + rank * kW4Threads; i < m * a.channels; i += split * kW4Threads) {
      const int tok = i / a.channels, ch = i % a.channels, n = n0 + ch;
      if (n >= a.N) continue;
      const float xsc = a.x_scale ? a.x_scale[chunk + tok] : 1.f;
      float v;
      if (a.up) {
        const int r = (ch / 16) * 32 + ch % 16;
        const float gate = total(tok, r) * xsc, up = total(tok, r + 16) * xsc;
        v = gate / (1.f + expf(-gate)) * up;
      } else {
        v = total(tok, ch) * xsc;
      }
      const int64_t at = (int64_t)(chunk + tok) * a.N + n;
      if (a.out_dtype == MOE_DT_BF16)
        static_cast<__nv_bfloat16*>(a.out)[at] = from_f<__nv_bfloat16>(v);
      else if (a.out_dtype == MOE_DT_FP16)
        static_cast<__half*>(a.out)[at] = from_f<__half>(v);
      else
        static_cast<float*>(a.out)[at] = v;
    }
    // the next chunk (or the exit) must not overtake a reader of this part
    if (split > 1)
      cluster_sync_all();
    else
      __syncthreads();
  }
}

template <typename X, int NB, int GS, bool ZEROS>
void launch_as(const Launch& L, const W4Args& a, int split) {
  const int smem = W4Smem<X, NB>::bytes(panel_groups(a.group, a.K), ZEROS);
  // the kernel's largest shared memory on any call: groups of 32 with zeros
  constexpr int kSlotX = std::is_same<X, XBf16>::value ? 0 : std::is_same<X, XFp16>::value ? 1 : 2;
  constexpr int kSlotIndex = ((kSlotX * 2 + NB - 1) * 3 + GS / 2) * 2 + ZEROS;
  static_assert(kSlotIndex < kAttrW4Slots, "one slot for each variant");
  set_smem_attr_once(reinterpret_cast<const void*>(w4_gemv_kernel<X, NB, GS, ZEROS>),
                     W4Smem<X, NB>::bytes(kW4Panel / (32 * GS), ZEROS), kAttrW4Base + kSlotIndex);
  const dim3 grid(split, (a.N + a.channels - 1) / a.channels, a.E);
  launch_begin(L, MOE_K_W4);
  launch_kernel_cluster(w4_gemv_kernel<X, NB, GS, ZEROS>, grid, dim3(split), dim3(kW4Threads), smem,
                        L.stream, a);
  launch_end(L, MOE_K_W4);
}
template <typename X, int NB, int GS>
void launch_zeros(const Launch& L, const W4Args& a, int split) {
  if (a.z[0])
    launch_as<X, NB, GS, true>(L, a, split);
  else
    launch_as<X, NB, GS, false>(L, a, split);
}
template <typename X, int NB>
void launch_group(const Launch& L, const W4Args& a, int split) {
  if (a.group == 32)
    launch_zeros<X, NB, 1>(L, a, split);
  else if (a.group == 64)
    launch_zeros<X, NB, 2>(L, a, split);
  else
    launch_zeros<X, NB, 4>(L, a, split);
}
template <typename X>
void launch_w4(const Launch& L, const W4Args& a) {
  const int tiles = (a.N + a.channels - 1) / a.channels;
  const int panels = (a.K + kW4Panel - 1) / kW4Panel;
  const int64_t ctas = (int64_t)tiles * std::min(a.E, a.R);  // experts with rows, at most
  int split = 1;
  while (2 * split <= std::min(kW4MaxSplit, panels) && ctas * split < 2 * L.num_sms) split *= 2;
  // rows an expert has on average; more than eight go as two blocks a pass
  if ((int64_t)a.R > 8LL * a.E)
    launch_group<X, 2>(L, a, split);
  else
    launch_group<X, 1>(L, a, split);
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" moe_status moe_w4_gemv(int32_t n_experts, int32_t N, int32_t K, int32_t group, int32_t R,
                                  const int32_t* offsets, int32_t x_dtype, const void* x,
                                  const float* x_scale, const void* w, const void* w_up,
                                  int32_t scale_dtype, const void* scales, const void* scales_up,
                                  const uint8_t* zeros, const uint8_t* zeros_up, int32_t out_dtype,
                                  void* out, moe_stream_t stream) {
  if (n_experts < 1 || N < 1 || K < 32 || K % 32 || R < 0) return MOE_ERR_INVALID_ARG;
  if (group != 0 && group != 32 && group != 64 && group != 128) return MOE_ERR_INVALID_ARG;
  if (group > 0 && K % group) return MOE_ERR_INVALID_ARG;
  if (x_dtype != MOE_DT_BF16 && x_dtype != MOE_DT_FP16 && x_dtype != MOE_DT_INT8)
    return MOE_ERR_INVALID_ARG;
  if (scale_dtype < MOE_DT_BF16 || scale_dtype > MOE_DT_FP32 || out_dtype < MOE_DT_BF16 ||
      out_dtype > MOE_DT_FP32)
    return MOE_ERR_INVALID_ARG;
  if (!offsets && n_experts != 1) return MOE_ERR_INVALID_ARG;
  if ((w_up != nullptr) != (scales_up != nullptr) || (zeros_up && !w_up) ||
      (w_up && (zeros != nullptr) != (zeros_up != nullptr)))
    return MOE_ERR_INVALID_ARG;
  if (n_experts > kW4MaxExperts || N > (1 << 22) || K > (1 << 22)) return MOE_ERR_UNSUPPORTED;
  if (R == 0) return MOE_OK;
  if (!x || !w || !scales || !out) return MOE_ERR_INVALID_ARG;
  if ((x_dtype == MOE_DT_INT8) != (x_scale != nullptr)) return MOE_ERR_INVALID_ARG;
  if (misaligned16(offsets, x, x_scale, w, w_up, scales, scales_up, zeros, zeros_up, out))
    return MOE_ERR_ALIGNMENT;
  W4Args a{};
  a.offsets = offsets;
  a.x = x;
  a.x_scale = x_scale;
  a.w[0] = static_cast<const uint8_t*>(w);
  a.w[1] = static_cast<const uint8_t*>(w_up);
  a.s[0] = scales;
  a.s[1] = scales_up;
  a.z[0] = zeros;
  a.z[1] = zeros_up;
  a.out = out;
  a.E = n_experts;
  a.N = N;
  a.K = K;
  a.R = R;
  a.group = group > 0 ? group : K;
  a.groups = K / a.group;
  a.up = w_up != nullptr;
  a.channels = a.up ? kW4Rows / 2 : kW4Rows;
  a.scale_dtype = scale_dtype;
  a.out_dtype = out_dtype;
  Launch L;
  const moe_status s = open_launch(stream, &L);
  if (s != MOE_OK) return s;
  if (x_dtype == MOE_DT_BF16)
    launch_w4<XBf16>(L, a);
  else if (x_dtype == MOE_DT_FP16)
    launch_w4<XFp16>(L, a);
  else
    launch_w4<XInt8>(L, a);
  return launch_status_take();
}
