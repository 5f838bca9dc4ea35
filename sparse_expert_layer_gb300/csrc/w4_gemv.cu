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
//
// 56 experts' gate and up (5120 -> 1536, groups of 128, 192 rows) take 109 us,
// 4.2 TB/s, 62% of the copy rate.  No unit is full: the schedulers issue in 62% of
// the cycles, the half-rate integer pipe is busy in 57%, the tensor pipe in 24%,
// with four warps a scheduler (128 registers a thread).  The same loads without
// the arithmetic take 78 us, so what is lost is overlap of the two.  Half of the
// instructions take nibbles apart: eleven for eight weights in bf16 (nine in
// fp16), seven of them on the integer pipe; the rest permutes x, forms addresses
// and applies scales.  Leaving the subtraction of z to a sum of x by another MMA
// was no faster (111 us) and less exact.
//
// 14 experts' down (2048 -> 7168, groups of 32 with zero points, 37 rows) take 45
// us, 40%, and fill less still (issue 50%, integer pipe 37%, tensor pipe 12%): a
// CTA has four panels beside its start and the adding of its parts, and 784 CTAs on
// 304 slots are 2.6 rounds that run as three.  With zero points the registers do
// not suffice and 56 to 104 bytes a thread are spilled, up to 24 without.
#include <math.h>

#include <algorithm>

#include "rows.cuh"
#include "w4_plan.h"

namespace moe {

namespace {

constexpr int kW4MaxExperts = 4096;
constexpr int kW4Warps = 8;
constexpr int kW4Threads = 32 * kW4Warps;
constexpr int kW4Panel = 512;              // K of a panel of x and scales
constexpr int kW4Stage = 128;              // K of a ring stage
constexpr int kW4RowBytes = kW4Stage / 2;  // 64: four 16-byte pieces, swizzled
constexpr int kW4StageBytes = 32 * kW4RowBytes;
constexpr int kW4XStride = kW4Panel * 2 + 64;  // token rows 64 bytes apart modulo the banks
constexpr int kW4RedStride = kW4Rows + 4;

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
  // shared memory of the scales and zero points of a panel: bytes between rows,
  // and the copy unit (a power of two of at least 4 bytes)
  int sstride, zstride, sunit, zunit;
  int64_t sbytes, zbytes;  // of the whole tensors
};

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
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};
struct MmaFp16 {
  static constexpr uint32_t kMagic = 0x64006400u;  // 1024
  // a / 16 + b
  static __device__ __forceinline__ uint32_t sixteenth(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(0x2c002c00u), "r"(b));
    return d;
  }
  static __device__ __forceinline__ uint32_t sub(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  static __device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                             uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
};

__device__ __forceinline__ float lds_f32(uint32_t at) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint16_t lds_u16(uint32_t at) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}

// N consecutive 16-bit values from shared memory, in one load where they are
// aligned to their size: two a word.
template <int N>
__device__ __forceinline__ void load_halves(bool whole, uint32_t at, uint32_t (&w)[(N + 1) / 2]) {
  if (N > 1 && whole) {
    if constexpr (N == 4)
      asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at) : "memory");
    else
      asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(at) : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 2)
      w[i / 2] = lds_u16(at + 2 * i) | (i + 1 < N ? (uint32_t)lds_u16(at + 2 * i + 2) << 16 : 0u);
  }
}
// N consecutive scales of four rows each, as fp32.
template <typename T, int N>
__device__ __forceinline__ void load_scales(bool whole, const uint32_t (&at)[4], uint32_t off,
                                            float (&v)[4][N]) {
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[r][i] = lds_f32(at[r] + off + 4 * i);
    } else {
      uint32_t w[(N + 1) / 2];
      load_halves<N>(whole, at[r] + off, w);
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        const float2 f = unpack2<T>(w[i / 2]);
        v[r][i] = f.x;
        if (i + 1 < N) v[r][i + 1] = f.y;
      }
    }
  }
}
// N consecutive zero points, one a byte.
template <int N>
__device__ __forceinline__ uint32_t load_zeros(bool whole, uint32_t at) {
  uint32_t v = 0u;
  if (N == 4 && whole) {
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v |= lds_u8(at + i) << (8 * i);
  }
  return v;
}

// The x types: bytes of a channel, the MMA type, where 16-byte piece i of token
// row r lies in a panel, and a thread's operands of one 32-wide step: its eight
// channels k0 .. k7 as the words (k0,k4) (k1,k5) (k2,k6) (k3,k7), the order in
// which the nibbles of a weight word pair up.
struct XBf16 {
  using Mma = MmaBf16;
  static constexpr int kBytes = 2;
  static constexpr int kRow = kW4Panel * 2;
  // every second row has its 64-byte halves swapped: two rows cover the banks
  static __device__ __forceinline__ uint32_t piece(int r, int i) {
    return r * kRow + ((i ^ ((r & 1) * 4)) * 16);
  }
  static __device__ __forceinline__ void operands(uint32_t panel, int r, int c, int step,
                                                  uint32_t (&b)[4]) {
    uint32_t x, y, z, w;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(x), "=r"(y), "=r"(z), "=r"(w)
                 : "r"(panel + piece(r, step * 4 + c))
                 : "memory");
    b[0] = __byte_perm(x, z, 0x5410);
    b[1] = __byte_perm(x, z, 0x7632);
    b[2] = __byte_perm(y, w, 0x5410);
    b[3] = __byte_perm(y, w, 0x7632);
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
  static constexpr int kRow = kW4Panel + 32;  // four rows cover the banks
  static __device__ __forceinline__ uint32_t piece(int r, int i) { return r * kRow + i * 16; }
  static __device__ __forceinline__ void operands(uint32_t panel, int r, int c, int step,
                                                  uint32_t (&b)[4]) {
    uint32_t lo, hi;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                 : "=r"(lo), "=r"(hi)
                 : "r"(panel + r * kRow + step * 32 + c * 8)
                 : "memory");
    lo ^= 0x80808080u;
    hi ^= 0x80808080u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // bytes (k_i, k_{i+4}) into the low bytes of two halves under 0x64
      const uint32_t both = __byte_perm(lo, hi, i | ((4 + i) << 4));
      b[i] = MmaFp16::sub(__byte_perm(both, 0x64646464u, 0x4140), 0x64806480u);
    }
  }
};

// (w & mask) | magic in one instruction; the compiler alone makes it two.
__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t mask, uint32_t magic) {
  uint32_t v;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(v) : "r"(w), "r"(mask), "r"(magic));
  return v;
}
// A weight word holds channels k0 .. k7, a nibble each, k0 lowest.  Pair i is
// (q(k_i) - z, q(k_{i+4}) - z) in 16 bits each, exact.  zero[0] holds magic + z;
// fp16 has room for a nibble four bits up as well (1024 + 16 q, exact), which
// saves two of three shifts: zero[1] holds -(64 + z) for those.
template <typename M>
__device__ __forceinline__ void dequant(uint32_t w, const uint32_t (&zero)[2], uint32_t (&p)[4]) {
  if constexpr (std::is_same<M, MmaFp16>::value) {
    const uint32_t v = w >> 8;
    p[0] = M::sub(and_or(w, 0x000f000fu, M::kMagic), zero[0]);
    p[1] = M::sixteenth(and_or(w, 0x00f000f0u, M::kMagic), zero[1]);
    p[2] = M::sub(and_or(v, 0x000f000fu, M::kMagic), zero[0]);
    p[3] = M::sixteenth(and_or(v, 0x00f000f0u, M::kMagic), zero[1]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      p[i] = M::sub(and_or(w >> (4 * i), 0x000f000fu, M::kMagic), zero[0]);
  }
}

// Shared memory: the warps' rings, then two panels of x, scales and zero points;
// the parts of a sum lie over the rings once those are drained.  Two CTAs fit an
// SM, except for 16-bit x with fp32 scales of groups of 32 (w4_memory).  (A variant
// for eight token rows with 80 registers and three CTAs an SM was no faster: 32.0
// against 30.3 us for 38912 x 6144.)
constexpr int kW4MaxRows = 16;  // token rows of one pass over the weights
constexpr int kW4Stages = 4;
constexpr int kW4Ring = kW4Warps * kW4Stages * kW4StageBytes;
static_assert(kW4MaxRows * kW4RedStride * 4 <= kW4Ring, "the parts fit over the rings");
template <typename X>
constexpr int kW4XPanel = kW4MaxRows* X::kRow;

// One thread's part in copying the scales (or zero points) of a weight row.
struct W4Groups {
  const unsigned char* from;  // its first unit of the next panel
  uint32_t dst;               // where that goes in the first buffer
  int unit, step;             // bytes of a unit, and from panel to panel
  int panel, end, whole;      // bytes from `from` to the panel's, row's, tensor's end
};

// What a CTA works on.
struct W4Tile {
  int e, n0, rank, split;
  int p0, p1;  // panels of K
};

// One pass over the tile's weights for m <= 8 * NB token rows from `row` on.
// GS: 32-wide K steps that share a scale (group 32: 1, 64: 2, 128 or a whole
// row: 4).
template <typename X, int NB, int GS, bool ZEROS>
__device__ __forceinline__ void w4_pass(const W4Args& a, const W4Tile& t, int row, int m,
                                        unsigned char* smem) {
  using M = typename X::Mma;
  constexpr int kGroups = 16 / GS;  // of a panel
  constexpr int kStages = kW4Stages, kRing = kW4Ring, kXPanel = kW4XPanel<X>;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int nw = warp % 4, kw = warp / 4;
  const int g = lane / 4, c = lane % 4;
  const uint32_t base = smem_u32(smem);
  const uint32_t xs = base + kRing;
  const uint32_t scales = xs + 2 * kXPanel;
  const uint32_t zeros = scales + 2 * kW4Rows * a.sstride;
  const uint32_t ring = base + warp * kStages * kW4StageBytes;

  // Weight row i (0 .. 127) of the CTA belongs to warp tile i / 32; with a second
  // matrix rows 0-15 of a warp tile are the first's, 16-31 the second's, of 16
  // channels.  Rows past N stand for channel N - 1: they are not stored.
  auto row_channel = [&](int i) {
    return min(a.up ? t.n0 + (i / 32) * 16 + i % 16 : t.n0 + i, a.N - 1);
  };

  // Stage q of this warp: 128 channels from p0 * 512 + q * 256 + kw * 128 on, two
  // stages a panel.  The lane copies 16-byte piece lane % 4 of rows i * 8 +
  // lane / 4; pieces of a row are swizzled so that neither these writes nor
  // ldmatrix meet a bank twice.  Pieces past K are left as they are: whatever codes
  // lie there meet zeros of x.
  const int half = a.K / 2;  // bytes of a weight row
  const uint8_t* wp[4];      // the lane's pieces of the next stage to be loaded
#pragma unroll
  for (int i = 0; i < 4; ++i)
    wp[i] = a.w[a.up ? i / 2 : 0] +
            ((int64_t)t.e * a.N + row_channel(nw * 32 + i * 8 + lane / 4)) * half +
            (t.p0 * kW4Panel + kw * kW4Stage) / 2 + (lane % 4) * 16;
  // bytes from there to the end of the row, or of this CTA's range
  int wleft = min(half, t.p1 * (kW4Panel / 2)) -
              ((t.p0 * kW4Panel + kw * kW4Stage) / 2 + (lane % 4) * 16);
  const uint32_t fill0 = ring + (lane / 4) * kW4RowBytes + (((lane % 4) ^ ((lane / 8) % 4)) * 16);
  uint32_t fill = 0, use = 0;  // the ring stages to be filled and to be used next
  auto next = [](uint32_t& at) {
    at = at == (kStages - 1) * kW4StageBytes ? 0 : at + kW4StageBytes;
  };
  auto load_stage = [&]() {
    if (wleft > 0)
#pragma unroll
      for (int i = 0; i < 4; ++i) cp_async16(fill0 + fill + i * 8 * kW4RowBytes, wp[i]);
    cp_async_commit();
    wleft -= kW4Panel / 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) wp[i] += kW4Panel / 4;
    next(fill);
  };

  // A panel of x, scales and zero points into buffer `buf`, by all threads; the
  // pointers go on from panel to panel.  x: 16-byte pieces of the present token
  // rows, zeros past K.  Scales and zero points: thread tid takes every second
  // copy unit of row tid % 128, from the last unit boundary at or before the
  // row's first group (rows of odd lengths start inside a unit).
  constexpr int kPieces = kW4Panel * X::kBytes / 16;  // of a token row
  constexpr int kTokStep = kW4Threads / kPieces;
  const int tok0 = tid / kPieces;
  int kx = t.p0 * kW4Panel + (tid % kPieces) * (16 / X::kBytes);
  const unsigned char* xp =
      static_cast<const unsigned char*>(a.x) + ((int64_t)(row + tok0) * a.K + kx) * X::kBytes;
  const int es = a.scale_dtype == MOE_DT_FP32 ? 4 : 2;
  auto first_group = [&](int i) {  // row i's first group
    return ((int64_t)t.e * a.N + row_channel(i)) * a.groups;
  };
  auto groups_of = [&](const void* src, int bytes, int unit, int64_t tensor, uint32_t dst) {
    W4Groups r;
    const int64_t first = first_group(tid % kW4Rows) * bytes, at = first & ~(int64_t)(unit - 1);
    const int64_t skip = a.groups > 1 ? (int64_t)t.p0 * kGroups * bytes : 0;
    const int mine = tid / kW4Rows * unit;  // every second unit of the row
    r.from = static_cast<const unsigned char*>(src) + at + skip + mine;
    r.dst = dst + mine;
    r.unit = unit;
    r.step = a.groups > 1 ? kGroups * bytes : 0;
    r.panel = (int)(first - at) + kGroups * bytes - mine;
    r.end = (int)(first - at) + (int)(a.groups * bytes - skip) - mine;
    r.whole = (int)min(tensor - at - skip - mine, (int64_t)INT32_MAX);
    return r;
  };
  auto load_groups = [&](W4Groups& r, uint32_t off) {
    const int end = min(r.end, r.panel);
    for (int i = 0; i < end; i += 2 * r.unit) {
      if (i + r.unit <= r.whole) {
        cp_async_unit(r.dst + off + i, r.from + i, r.unit);
      } else {  // the tensor ends inside its last word
        for (int j = i; j < r.whole; ++j)
          asm volatile("st.shared.u8 [%0], %1;" ::"r"(r.dst + off + j), "r"((uint32_t)r.from[j])
                       : "memory");
      }
    }
    r.from += r.step;
    r.end -= r.step;
    r.whole -= r.step;
  };
  const int smat = a.up ? (tid % kW4Rows / 16) % 2 : 0;
  W4Groups sg = groups_of(a.s[smat], es, a.sunit, a.sbytes, scales + tid % kW4Rows * a.sstride);
  W4Groups zg{};
  if constexpr (ZEROS)
    zg = groups_of(a.z[smat], 1, a.zunit, a.zbytes, zeros + tid % kW4Rows * a.zstride);
  auto load_panel = [&](int buf) {
    const bool in = kx < a.K;
#pragma unroll
    for (int i = 0; i < NB * 8 / kTokStep; ++i)
      if (tok0 + i * kTokStep < m)
        cp_async16_or_zero(
            xs + buf * kXPanel + X::piece(tok0 + i * kTokStep, tid % kPieces),
            in ? xp + (int64_t)i * kTokStep * a.K * X::kBytes
               : static_cast<const unsigned char*>(a.x),
            in);
    kx += kW4Panel;
    xp += kW4Panel * X::kBytes;
    load_groups(sg, buf * kW4Rows * a.sstride);
    if constexpr (ZEROS) load_groups(zg, buf * kW4Rows * a.zstride);
  };
  // Where this thread's four weight rows have the scales and zero points of its
  // first stage of a panel.  kGps groups a stage, in one load where rows are whole
  // numbers of them.
  constexpr int kGps = 4 / GS;
  const bool one = a.groups == 1;
  const bool whole = a.groups % kGps == 0;
  uint32_t srow[4], zrow[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = nw * 32 + g + i * 8;
    srow[i] = scales + r * a.sstride + ((uint32_t)first_group(r) * es & (a.sunit - 1)) +
              (one ? 0 : kw * kGps * es);
    if constexpr (ZEROS)
      zrow[i] = zeros + r * a.zstride + ((uint32_t)first_group(r) & (a.zunit - 1)) +
                (one ? 0 : kw * kGps);
  }

  // absent token rows are zero in both panels
  for (int i = m * kPieces + tid; i < NB * 8 * kPieces; i += kW4Threads)
#pragma unroll
    for (int b = 0; b < 2; ++b)
      *reinterpret_cast<uint4*>(smem + kRing + b * kXPanel +
                                X::piece(i / kPieces, i % kPieces)) = make_uint4(0u, 0u, 0u, 0u);

  float acc[2][NB][4] = {};
  if (t.p0 < t.p1) load_panel(0);  // completes with the first stage
#pragma unroll
  for (int q = 0; q < kStages - 1; ++q) load_stage();

  // One stage: half HALF of panel p, whose x and scales are in buffer `buf`.
  auto stage = [&](auto which, int p, int buf) {
    constexpr int kHalf = decltype(which)::value;
    if constexpr (kHalf == 0) {
      // The panel came with the stage after this one (the first panel with the
      // first); everybody is done with the panel before, whose buffer the next
      // one takes.
      cp_async_wait<kStages - 3>();
      __syncthreads();
      if (p + 1 < t.p1) load_panel(buf ^ 1);
    } else {
      cp_async_wait<kStages - 2>();
      __syncwarp();
    }
    load_stage();
    const uint32_t at = use;
    next(use);
    const int k0 = p * kW4Panel + kHalf * (kW4Panel / 2) + kw * kW4Stage;
    if (k0 >= a.K) return;  // warp-uniform; no scales there
    const uint32_t st = ring + at + lane * kW4RowBytes;
    const uint32_t xb = xs + buf * kXPanel;

    // the operands of a 32-wide step, loaded a step ahead of their use: weights of
    // the first tile's rows g, g + 8 and the second's, and x
    uint32_t wn[4], bn[NB][4];
    auto load_step = [&](int s) {
      ldmatrix_x4(st + ((s ^ ((lane / 2) % 4)) * 16), wn);
#pragma unroll
      for (int b = 0; b < NB; ++b) X::operands(xb, b * 8 + g, c, kHalf * 8 + kw * 4 + s, bn[b]);
    };
    load_step(0);

    // the stage's scales and zero points, as they are
    float sv[4][kGps];
    uint32_t zv[4];
    const uint32_t so = buf * kW4Rows * a.sstride + (one ? 0 : kHalf * 2 * kGps * es);
    if (a.scale_dtype == MOE_DT_BF16)
      load_scales<__nv_bfloat16, kGps>(whole, srow, so, sv);
    else if (a.scale_dtype == MOE_DT_FP16)
      load_scales<__half, kGps>(whole, srow, so, sv);
    else
      load_scales<float, kGps>(whole, srow, so, sv);
    if constexpr (ZEROS)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        zv[i] = load_zeros<kGps>(whole, zrow[i] + buf * kW4Rows * a.zstride +
                                            (one ? 0 : kHalf * 2 * kGps)) & 0x1f1f1f1fu;
#pragma unroll
    for (int s0 = 0; s0 < 4; s0 += GS) {
      if (k0 + s0 * 32 >= a.K) break;
      uint32_t zc[4][2];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        zc[i][0] = ZEROS ? __byte_perm(zv[i], M::kMagic >> 8, 0x4040 + (s0 / GS) * 0x0101)
                         : M::kMagic + 0x00080008u;
        // fp16: 960 - (1024 + z); bf16 has no use for it
        zc[i][1] = ZEROS ? M::sub(0x63806380u, zc[i][0]) : 0xd480d480u;
      }
      float part[2][NB][4] = {};
#pragma unroll
      for (int s = s0; s < s0 + GS; ++s) {
        uint32_t wv[4], bf[NB][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          wv[i] = wn[i];
#pragma unroll
          for (int b = 0; b < NB; ++b) bf[b][i] = bn[b][i];
        }
        if (s < 3) load_step(s + 1);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          uint32_t lo[4], hi[4];  // rows g and g + 8
          dequant<M>(wv[2 * u], zc[2 * u], lo);
          dequant<M>(wv[2 * u + 1], zc[2 * u + 1], hi);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t af[4] = {lo[2 * i], hi[2 * i], lo[2 * i + 1], hi[2 * i + 1]};
#pragma unroll
            for (int b = 0; b < NB; ++b) M::mma(part[u][b], af, bf[b][2 * i], bf[b][2 * i + 1]);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            acc[u][b][j] = fmaf(sv[2 * u + j / 2][s0 / GS], part[u][b][j], acc[u][b][j]);
    }
  };
  for (int p = t.p0; p < t.p1; ++p) {
    stage(std::integral_constant<int, 0>{}, p, (p - t.p0) & 1);
    stage(std::integral_constant<int, 1>{}, p, (p - t.p0) & 1);
  }
  cp_async_wait<0>();
  __syncthreads();

  // add the two K halves, then the cluster's parts, in a fixed order
  float* red = reinterpret_cast<float*>(smem);
  auto red_at = [&](int u, int b, int j) -> float& {
    const int tok = b * 8 + 2 * c + (j & 1), r = nw * 32 + u * 16 + g + (j >> 1) * 8;
    return red[tok * kW4RedStride + r];
  };
  if (kw == 1) {
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int j = 0; j < 4; ++j) red_at(u, b, j) = acc[u][b][j];
  }
  __syncthreads();
  if (kw == 0) {
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int j = 0; j < 4; ++j) red_at(u, b, j) += acc[u][b][j];
  }
  if (t.split > 1)
    cluster_sync_all();
  else
    __syncthreads();
  auto total = [&](int tok, int r) {
    if (t.split == 1) return red[tok * kW4RedStride + r];
    const uint32_t at = base + (tok * kW4RedStride + r) * 4;
    float v[kW4MaxSplit], sum = 0.f;
#pragma unroll
    for (int q = 0; q < kW4MaxSplit; ++q)
      if (q < t.split) v[q] = ld_cluster_f32(mapa_shared(at, q));
#pragma unroll
    for (int q = 0; q < kW4MaxSplit; ++q)
      if (q < t.split) sum += v[q];
    return sum;
  };
  for (int i = tid + t.rank * kW4Threads; i < m * a.channels; i += t.split * kW4Threads) {
    const int tok = i / a.channels, ch = i % a.channels, n = t.n0 + ch;
    if (n >= a.N) continue;
    const float xsc = a.x_scale ? a.x_scale[row + tok] : 1.f;
    float v;
    if (a.up) {
      const int r = (ch / 16) * 32 + ch % 16;
      const float gate = total(tok, r) * xsc, up = total(tok, r + 16) * xsc;
      v = gate / (1.f + expf(-gate)) * up;
    } else {
      v = total(tok, ch) * xsc;
    }
    const int64_t at = (int64_t)(row + tok) * a.N + n;
    if (a.out_dtype == MOE_DT_BF16)
      static_cast<__nv_bfloat16*>(a.out)[at] = from_f<__nv_bfloat16>(v);
    else if (a.out_dtype == MOE_DT_FP16)
      static_cast<__half*>(a.out)[at] = from_f<__half>(v);
    else
      static_cast<float*>(a.out)[at] = v;
  }
  // the next pass (or the exit) must not overtake a reader of these parts
  if (t.split > 1)
    cluster_sync_all();
  else
    __syncthreads();
}

template <typename X, int GS, bool ZEROS>
__global__ void __launch_bounds__(kW4Threads, 2) w4_gemv_kernel(W4Args a) {
  pdl_enter();
  extern __shared__ __align__(128) unsigned char smem[];
  W4Tile t;
  t.e = blockIdx.z;
  t.n0 = blockIdx.y * a.channels;
  t.rank = blockIdx.x;
  t.split = gridDim.x;
  int row0 = 0, row1 = a.R;
  if (a.offsets) {  // offsets are data: stay inside the R rows whatever they hold
    row0 = min(max(a.offsets[t.e], 0), a.R);
    row1 = min(max(a.offsets[t.e + 1], row0), a.R);
  }
  const int panels = (a.K + kW4Panel - 1) / kW4Panel;
  const int per = (panels + t.split - 1) / t.split;
  t.p0 = min(panels, t.rank * per);
  t.p1 = min(panels, t.p0 + per);
  // the whole cluster sees the same rows, so its barriers match
  while (row0 < row1) {
    const int m = min(row1 - row0, kW4MaxRows);
    if (m > 8)
      w4_pass<X, 2, GS, ZEROS>(a, t, row0, m, smem);
    else
      w4_pass<X, 1, GS, ZEROS>(a, t, row0, m, smem);
    row0 += m;
  }
}

template <typename X, int GS, bool ZEROS>
void launch_as(const Launch& L, W4Args a) {
  const int es = a.scale_dtype == MOE_DT_FP32 ? 4 : 2;
  constexpr int kFixed = kW4Ring + 2 * kW4XPanel<X>;
  const W4Memory mem = w4_memory(kFixed, a.groups, 16 / GS, es, ZEROS);
  a.sunit = mem.sunit;
  a.sstride = mem.sstride;
  a.sbytes = (int64_t)a.E * a.N * a.groups * es;
  if (ZEROS) {
    a.zunit = mem.zunit;
    a.zstride = mem.zstride;
    a.zbytes = (int64_t)a.E * a.N * a.groups;
  }
  const int row_tiles = (a.N + a.channels - 1) / a.channels;
  const int experts = std::min(a.E, a.R);  // with rows, at most
  const int split = w4_choose_split((int64_t)row_tiles * experts,
                                    (a.K + kW4Panel - 1) / kW4Panel, L.num_sms, mem.per_sm);
  // at most: fp32 scales of groups of 32 and their zero points
  constexpr int kMost = kFixed + 2 * kW4Rows * (96 + 48);
  constexpr int kSlotX = std::is_same<X, XBf16>::value ? 0 : std::is_same<X, XFp16>::value ? 1 : 2;
  constexpr int kSlotIndex = (kSlotX * 3 + GS / 2) * 2 + ZEROS;
  static_assert(kSlotIndex < kAttrW4Slots, "one slot for each variant");
  set_smem_attr_once(reinterpret_cast<const void*>(w4_gemv_kernel<X, GS, ZEROS>), kMost,
                     kAttrW4Base + kSlotIndex);
  const dim3 grid(split, row_tiles, a.E);
  launch_begin(L, MOE_K_W4);
  launch_kernel_cluster(w4_gemv_kernel<X, GS, ZEROS>, grid, dim3(split), dim3(kW4Threads),
                        mem.bytes, L.stream, a);
  launch_end(L, MOE_K_W4);
}

template <typename X, int GS>
void launch_zeros(const Launch& L, const W4Args& a) {
  if (a.z[0])
    launch_as<X, GS, true>(L, a);
  else
    launch_as<X, GS, false>(L, a);
}
template <typename X>
void launch_w4(const Launch& L, const W4Args& a) {
  if (a.group == 32)
    launch_zeros<X, 1>(L, a);
  else if (a.group == 64)
    launch_zeros<X, 2>(L, a);
  else
    launch_zeros<X, 4>(L, a);
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
  // 32-bit offsets inside one expert's matrix; at most 65535 row tiles
  if (n_experts > kW4MaxExperts || N > (1 << 21) || K > (1 << 22) ||
      (int64_t)N * (K / 2) > INT32_MAX)
    return MOE_ERR_UNSUPPORTED;
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
  a.group = group;
  a.groups = group > 0 ? K / group : 1;
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
