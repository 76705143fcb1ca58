// How the attention over a paged cache (bfly_attend.hip) is cut into workgroups,
// and the scratch that takes: plain C++, of the sizes of a call only.
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>

namespace bfly {

constexpr int kAttendStep = 32;    // tokens of a wave's step: two tiles of 16
constexpr int kAttendHeads = 16;   // query heads a workgroup takes (matrix-core columns)

// Workgroups for the `share` query heads of a key-value head.
inline int attend_blocks(int share) { return (share + kAttendHeads - 1) / kAttendHeads; }

// The most tokens of a row that a call goes through: a window's first step may
// begin in front of it.
inline int attend_reach(int max_len, int window) {
  return window > 0 ? (int)std::min<int64_t>(max_len, (int64_t)window + kAttendStep - 1) : max_len;
}

// How a call's lengths, up to `reach`, are cut: into chunks, or not at all.
//   Up to 512 tokens (1024 where there are 128 items or more, each a row's
// key-value head) the second launch costs more than it spreads: 32 rows of 8
// heads of 1024 tokens int8 13.9 us in one chunk, 18.7 in 256s, 16.5 in 512s; 4
// rows of 512 tokens 7.3, in 128s 7.8, in 256s 8.8.
//   One row is as long as it is known to be: 512 workgroups (131072 tokens of
// e4m3 48.5 us; 55.0 with 1024, 61.8 with 256).
//   Rows of lengths that only the device knows: a card full of chunks as short
// as pays, since no workgroup may last much longer than the average.  128
// tokens, while there are at most 2048 workgroups (8 ragged rows of up to 1024:
// 8.0 us, in 256s 9.1, in 512s 11.0), up to 512 (32 rows of 4096, and ragged ones
// of up to 4096: 128 tokens 73.7 and 28.1 us, 256 64.4 and 21.7, 512 58.7 and
// 19.4, 1024 60.5 and 22.3; 64 ragged rows of up to 8192 int4: 256 58.2, 512
// 45.1, 1024 45.6, 2048 47.5), more where that would be above 8192 workgroups.
// 256 instead of 128 where a chunk's partial results, 16 heads of 256, are large
// (24 rows of a window of 2047: 15.2 for 16.5).
//   All this goes by the bound, not by the lengths: a bound far above them makes
// chunks long and workgroups few.  Sequences of 4096 tokens int8, 8 heads, with
// a bound of 4096, 32768 and 131072: one 8.4, 11.2 and 22.5 us, 32 of them 58.7,
// 58.0 and 67.9.
struct Cut {
  int chunk, splits;
};
constexpr int kOneChunk = 512, kAlone = 512, kMost = 8192;
inline Cut cut_of(int64_t rows, int64_t items, int share, int head_dim, int reach) {
  if (reach <= kOneChunk || (reach <= 2 * kOneChunk && items >= 128)) return {reach, 1};
  // a multiple of 128 tokens; no more than all (items times reach passes 32 bits)
  const auto whole = [&](int64_t v) {
    return (int)((std::min<int64_t>(v, reach) + 127) / 128 * 128);
  };
  const int least = std::min(share, kAttendHeads) * head_dim >= 2048 ? 256 : 128;
  // (rounded up without a sum, which passes 32 bits where both are 2^30)
  const auto splits = [&](int chunk) { return (reach - 1) / chunk + 1; };
  int chunk = least;
  if (rows == 1) {
    chunk = std::max(chunk, whole((items * reach + kAlone - 1) / kAlone));
  } else {
    while (chunk < 512 && items * splits(chunk) > 2048) chunk *= 2;
    if (items * splits(chunk) > kMost)
      chunk = std::max(chunk, whole((items * reach + kMost - 1) / kMost));
  }
  return {chunk, splits(chunk)};
}

// Bytes for the partial results of a call, over all windows.  Never falls with
// rows, heads, head_dim or max_len while kv_heads stays.
inline size_t attend_workspace_bytes(int64_t rows, int heads, int kv_heads, int head_dim,
                                     int max_len) {
  if (max_len <= kOneChunk) return 0;
  // no call has more than items + kMost chunks, of up to 16 heads each, nor
  // more than one for every 128 tokens
  const int share = heads / kv_heads, blocks = attend_blocks(share);
  const int64_t items = rows * kv_heads * blocks;
  const int64_t parts = std::min(rows * heads * ((max_len + 127) / 128),
                                 (items + kMost) * std::min(share, kAttendHeads));
  return (size_t)parts * (size_t)(head_dim + 4) * sizeof(float);
}

}  // namespace bfly
