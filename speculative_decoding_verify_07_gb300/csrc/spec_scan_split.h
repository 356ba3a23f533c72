// How spec_scan divides long rows, and the workspace that this takes (plain host arithmetic).
#pragma once

#include <stddef.h>

#include <algorithm>

namespace specv {

constexpr int kScanThreads = 128;      // of each half of a CTA
constexpr int kScanLane = 2;           // channels of a lane
constexpr int kScanTile = 16;          // tokens of a tile
constexpr int kScanCtas = 2;           // an SM
constexpr int kScanFine = 4, kScanLeast = 128;      // parts of a segment at most; no part is of fewer tokens

// A row's tokens where they are split into segments, and the workspace of such a call: each part's sum of delta by (row,
// part, channel), then by (row, part, channel, state) the state behind the part if it began with zeros, which
// scan_join_kernel turns into the state that enters it.  A segment has `fine` parts: scan_segment_kernel has fewer
// registers and takes more CTAs an SM.
struct ScanSplit {
  int segments, span, fine;            // span: tokens of a segment
  float* sums;
  float* states;
};

// CTAs a row (each: channels of a group).
inline int scan_blocks(int D, int each, int N) {
  const int ch = kScanThreads / (N / 4) * kScanLane;
  return (each + ch - 1) / ch * (D / each);
}

// Segments a row at most: one where there are CTAs for most SMs, otherwise as many as fill all of them once.  The first pass
// makes a split cost half as much again: 64 CTAs of 4096 tokens take 181 us in four segments, 247 in one, and a row of 512
// tokens 37 and 34; 256 CTAs of 2048 tokens took 220 us whole and 300 and more in two.
inline long long scan_want(long long ctas) { return ctas >= 100 ? 1 : std::max(1ll, 152 * kScanCtas / ctas); }

inline ScanSplit scan_split(int B, int T, int D, int each, int N) {
  const long long want = scan_want((long long)scan_blocks(D, each, N) * B);
  ScanSplit W = {};
  W.segments = (int)std::max(1ll, std::min(want, (long long)T / kScanLeast));
  W.fine = W.segments > 1 ? std::max(1, std::min(kScanFine, T / W.segments / kScanLeast)) : 1;
  const int unit = kScanTile * W.fine;
  W.span = (int)(((long long)T + (long long)W.segments * unit - 1) / ((long long)W.segments * unit) * unit);
  W.segments = (int)(((long long)T + W.span - 1) / W.span);
  return W;
}

// Parts of all rows that a call keeps.
inline long long scan_parts(const ScanSplit& W, int B) { return W.segments > 1 ? (long long)W.segments * W.fine * B : 0; }

// No division of up to B rows of up to T tokens has more, whatever its groups: one group has the fewest CTAs and so may have
// the most segments, but fewer segments may have more parts each, and fewer rows more segments.  Rows that are split have
// at most 152 kScanCtas segments for the CTAs of one, a segment at most kScanFine parts, and none of these is of fewer than
// kScanLeast tokens before segments are rounded up to whole tiles, which makes fewer of them.
inline long long scan_parts_most(int B, int T, int D, int N) {
  const int blocks = scan_blocks(D, D, N);
  return scan_want(blocks) > 1 ? std::min((long long)T / kScanLeast * B, 152ll * kScanCtas * kScanFine / blocks) : 0;
}

// Where the states lie in the workspace, and its bytes for so many parts.
inline size_t scan_states_at(long long parts, int D) { return ((size_t)parts * D * 4 + 255) / 256 * 256; }
inline size_t scan_bytes(long long parts, int D, int N) { return scan_states_at(parts, D) + (size_t)parts * D * N * 4; }

}  // namespace specv
