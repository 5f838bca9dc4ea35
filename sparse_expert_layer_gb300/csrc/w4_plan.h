// Launch rules of the 4-bit products (w4_gemv.cu), host code only.
#pragma once

#include <algorithm>
#include <cstdint>

namespace moe {

constexpr int kW4MaxSplit = 8;

// How many CTAs share a row tile's K: the split with the least time by a count
// of panels.  A CTA takes the time of its panels and of about two more to start
// and to add the parts.  Two CTAs fit an SM, and a cluster stays inside a GPC
// of 16 to 20 SMs, so larger clusters leave some slots empty; a device (or a
// partition) of fewer SMs counts as one GPC that holds at least one cluster.
inline int w4_choose_split(int64_t tiles, int panels, int num_sms) {
  const int gpcs = std::max(1, num_sms / 19), gpc_slots = 2 * std::min(18, num_sms);
  int best = 1;
  int64_t least = INT64_MAX;
  for (int split = 1; split <= std::min(kW4MaxSplit, panels); split *= 2) {
    const int64_t slots =
        split == 1 ? 2 * num_sms : std::max(split, gpcs * (gpc_slots / split * split));
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
