// Launch rules of the 4-bit products (w4_gemv.cu), host code only.
#pragma once

#include <algorithm>
#include <cstdint>

namespace moe {

constexpr int kW4MaxSplit = 8;
constexpr int kW4Rows = 128;  // weight rows of a CTA

// The shared memory of a CTA: `fixed` bytes of rings and panels of x, then two
// panels of scales and zero points.
struct W4Memory {
  int sunit, zunit;      // bytes of a copy unit of scales, of zero points
  int sstride, zstride;  // bytes between two weight rows
  int bytes;             // of the CTA
  int per_sm;            // CTAs that fit an SM
};

// The copy unit of rows of `row` bytes whose panels hold `panel` bytes: the
// widest that both are multiples of, or 4 with rows that start inside a unit.
inline int w4_copy_unit(int64_t row, int panel) {
  for (int u = 16; u > 4; u /= 2)
    if (row % u == 0 && panel % u == 0) return u;
  return 4;
}
// Bytes between rows: a row's panel, one unit more where rows may start inside a
// unit, and an odd number of units against bank conflicts.  Rows of at most 16
// bytes have none: eight of them lie side by side in the banks.  (Padded as well,
// zero points of 72 groups of 32 left room for one CTA an SM: 16 experts' 2304 ->
// 7168 took 74 us instead of 53.)
inline int w4_row_stride(int64_t row, int panel, int unit) {
  const int n = (panel + (row % unit ? unit : 0) + unit - 1) / unit;
  return (n % 2 == 0 && n * unit > 16 ? n + 1 : n) * unit;
}

inline W4Memory w4_memory(int fixed, int groups, int panel_groups, int scale_bytes, bool zeros) {
  W4Memory m{};
  const int64_t row = (int64_t)groups * scale_bytes;
  m.sunit = w4_copy_unit(row, panel_groups * scale_bytes);
  m.sstride = w4_row_stride(row, panel_groups * scale_bytes, m.sunit);
  if (zeros) {
    m.zunit = w4_copy_unit(groups, panel_groups);
    m.zstride = w4_row_stride(groups, panel_groups, m.zunit);
  }
  m.bytes = fixed + 2 * kW4Rows * (m.sstride + m.zstride);
  // an SM has 228 KB, a CTA takes 1 KB besides its own; registers allow two
  m.per_sm = 2 * (m.bytes + 1024) <= 228 * 1024 ? 2 : 1;
  return m;
}

// How many CTAs share a row tile's K: the split with the least time by a count
// of panels.  A CTA takes the time of its panels and of about two more to start
// and to add the parts.  `per_sm` CTAs fit an SM, and a cluster stays inside a GPC
// of 16 to 20 SMs, so larger clusters leave some slots empty; a device (or a
// partition) of fewer SMs counts as one GPC that holds at least one cluster.
inline int w4_choose_split(int64_t tiles, int panels, int num_sms, int per_sm = 2) {
  const int gpcs = std::max(1, num_sms / 19), gpc_slots = per_sm * std::min(18, num_sms);
  int best = 1;
  int64_t least = INT64_MAX;
  for (int split = 1; split <= std::min(kW4MaxSplit, panels); split *= 2) {
    const int64_t slots =
        split == 1 ? per_sm * num_sms : std::max(split, gpcs * (gpc_slots / split * split));
    const int64_t rounds = (tiles * split + slots - 1) / slots;
    const int64_t cost = rounds * ((panels + split - 1) / split + 2);
    if (cost < least) {
      least = cost;
      best = split;
    }
  }
  return best;
}

}  // namespace moe
