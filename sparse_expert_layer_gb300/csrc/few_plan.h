// Shared-memory plan of the layer for a few tokens (few_tokens.cu), host code only.
#pragma once

#include <algorithm>
#include <cstdint>

namespace moe {

constexpr int kFewMaxT = 8;
constexpr int kFewWarps = 16;
// Warps that share the K of one gate/up tile.  Two: the one token with 4-bit experts 69 us instead of
// 71 when this was measured, but eight with bf16 experts up to 358 instead of 353; eight: 76.
constexpr int kFewTeamWarps = 4;
constexpr int kFewTeams = kFewWarps / kFewTeamWarps;
constexpr int kFewSub = 2048;     // bytes of the weights of a ring stage: 16 rows of 128
constexpr int kFewMaxStages = 4;
constexpr int kFewSmem = 226 * 1024;  // dynamic; the kernel has a few words besides
constexpr int kFewUnitBytes = 8;
constexpr int kFewParts = 2 * kFewTeams * kFewTeamWarps * 16 * 8 * 4;  // bytes of the tiles' parts

// Layout of a CTA's shared memory: x, its block sums, units, rows of h, parts, rings.
struct FewPlan {
  int step_k;          // K of a stage: 256 four-bit or 64 sixteen-bit weights a row
  int xpitch;          // bytes between two tokens
  int block;           // K that shares a scale: 32, 64 or 128
  int hpitch, hrest;   // bytes between two rows of h there, to what 16-bit operands leave; 0:
                       // h does not fit
  int sum_at, unit_at, row_at, red_at, queue_at, ring_at;
  int swords, zwords;  // 4-byte words of scales and zero points a row has in a stage
  int s_eight, z_eight;  // bytes from a row's groups to those eight rows on
  int s_next, z_next;    // bytes from a block's scale (zero point) to the next one's, or 0
  int whole;             // rows are whole stages, so a stage's scales are aligned copies
  int sub_bytes;         // of a stage
  int stages;
  int bytes;           // of the CTA; stages < 2: does not fit
};

inline int few_round(int v, int to) { return (v + to - 1) / to * to; }

// The 4-byte words that hold n items of `size` bytes which start `size`-aligned in rows
// of `row` bytes.
inline int few_words(int n, int size, int64_t row) {
  const int bytes = n * size;
  return row % 4 == 0 && bytes % 4 == 0 ? bytes / 4 : (bytes + 4 - size + 3) / 4;
}

// units, rows: experts with tokens and rows of h, at most; inter: the longest row of h.
// group: 0 (a row), 32, 64, 128; rows_aligned: every row's scales (zero points) begin at a
// multiple of four bytes; two_terms: h is kept as two 16-bit numbers
inline FewPlan few_plan(int T, int H, int inter, int units, int rows, bool four_bits, int group,
                        int scale_bytes, bool zeros, bool rows_aligned_scales,
                        bool rows_aligned_zeros, bool whole, bool two_terms = true) {
  FewPlan p{};
  p.step_k = four_bits ? 256 : 64;
  p.block = four_bits ? (group ? group : 128) : 0;
  // two tokens' 64-byte pieces cover the banks
  p.xpitch = few_round(H, p.step_k) * 2 + 64;
  p.sum_at = T * p.xpitch;
  const int blocks = four_bits ? few_round(H, p.step_k) / p.block : 0;
  p.sub_bytes = kFewSub;
  if (four_bits) {
    const int n = group ? p.step_k / group : 1;
    p.swords = few_words(n, scale_bytes, rows_aligned_scales ? 4 : scale_bytes);
    p.zwords = zeros ? few_words(n, 1, rows_aligned_zeros ? 4 : 1) : 0;
    p.s_eight = 32 * p.swords;
    p.z_eight = 32 * p.zwords;
    p.s_next = group ? scale_bytes : 0;
    p.z_next = group ? 1 : 0;
    p.whole = whole;
    p.sub_bytes += few_round(16 * 4 * (p.swords + p.zwords), 16);
  }
  // x and its sums; later, where they leave four stages, all rows of h
  const int x_bytes = p.sum_at + blocks * kFewMaxT * 4;
  auto place = [&](int front) {
    p.unit_at = few_round(front, 16);
    p.row_at = p.unit_at + units * kFewUnitBytes;
    p.red_at = few_round(p.row_at + (units + 1 + rows) * 4, 16);
    p.queue_at = p.red_at + kFewParts;
    p.ring_at = few_round(p.queue_at + kFewTeams * 16 * 4, 128);
    p.stages = std::min(kFewMaxStages, (kFewSmem - p.ring_at) / (kFewWarps * p.sub_bytes));
  };
  const int64_t hpitch = (int64_t)few_round(inter, p.step_k) * 2 + 64;
  const int64_t h_bytes = rows * hpitch * (two_terms ? 2 : 1);
  if (h_bytes > 0 && h_bytes < kFewSmem) {
    place(std::max(x_bytes, (int)h_bytes));
    if (p.stages >= 4) {
      p.hpitch = (int)hpitch;
      p.hrest = (int)(rows * hpitch);
    }
  }
  if (p.hpitch == 0) place(x_bytes);
  p.bytes = p.ring_at + kFewWarps * p.stages * p.sub_bytes;
  // the parts of the down projection lie over the rings: 16 warps of 64 channels
  if (p.stages * p.sub_bytes < 64 * kFewMaxT * 4) p.stages = 0;
  return p;
}

}  // namespace moe
