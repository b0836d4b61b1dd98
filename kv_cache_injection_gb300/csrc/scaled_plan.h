// How a write into a scaled cache is spread over CTAs (scaled.cu).  Host code
// without CUDA, so that it is tested as it is.
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>

namespace isk {
namespace scaled {

// 128 threads and 32 KB of rows, five CTAs an SM: the steps of a CTA wait for one another, other CTAs fill the gaps (8000
// tokens 37 us, 51 with 256 threads and 64 KB, 45 with 128 threads and 16 KB).
constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kWindow = 30;              // tokens of a CTA, at most (a warp looks at them and a neighbour)
constexpr int kMaxGroups = 16;           // of a round
constexpr int kMaxRows = 128;            // of a round
constexpr int kDataBytes = 32768;        // of a round's rows: keys and values of the CTA's heads
constexpr int kMaxUnits = 8;             // a head's keys, or its values

// Rows of a round of a CTA with `heads_of` heads.
inline int rows_of_round(int heads_of, int D, int bytes) { return std::min(kMaxRows, kDataBytes / (2 * heads_of * D * bytes)); }

struct WritePlan {
  int window;                            // tokens of a CTA
  int heads_of;                          // heads of a CTA
  int rows;                              // of a round
  int share;                             // warps to a token's queries
  int64_t group_ctas, query_ctas;
  int64_t turns;                         // CTAs of either kind that take turns
  size_t smem;                           // bytes a CTA
};

// T tokens of Hq query and H KV heads (Hq 0: none) of D elements of `bytes` bytes, keys rotated or not.
inline WritePlan plan_write(int T, int Hq, int H, int D, int bytes, int block_size, int sms, bool rotate) {
  sms = std::max(1, sms);
  WritePlan w{};
  // Heads of a CTA: 4, 2 where a block's rows would not fit a round otherwise.
  w.heads_of = kMaxUnits / 2;
  while (w.heads_of > 2 && rows_of_round(w.heads_of, D, bytes) < std::min(block_size, kMaxRows)) w.heads_of /= 2;
  // Tokens of a CTA: one while every SM gets one, then up to 16 or a block.  Most tokens of a prompt begin no group, and CTAs
  // that end at once still hold up the others (8000 tokens with one a CTA: 74.6 us).
  w.window = std::min(std::min(kWindow, std::max(16, block_size)), std::max(1, T / sms));
  // Two heads too while all CTAs fit at once: one token 5.5 -> 5.0 us, 1276 moved tokens 7.9 -> 6.9, a prompt of 1600 16.9 ->
  // 15.3 (1000 single tokens 10.6 -> 11.3).
  const int64_t windows = ((int64_t)T + w.window - 1) / w.window, at_once = 5LL * sms;
  while (w.heads_of > 2 && windows * ((H + w.heads_of / 2 - 1) / (w.heads_of / 2)) <= at_once) w.heads_of /= 2;
  // One head where two heads' rows of a block do not fit a round, CTAs have several tokens and no more than two times as many
  // CTAs (most of which have no group then): 1276 tokens moved into blocks of 64 15.2 -> 9.7 us (8000 tokens would take 64,
  // not 56, and 100 single ones 6.2, not 5.4).
  if (w.heads_of == 2 && w.window > 1 && windows * H <= 2 * at_once && rows_of_round(2, D, bytes) < std::min(block_size, kMaxRows))
    w.heads_of = 1;
  w.group_ctas = windows * ((H + w.heads_of - 1) / w.heads_of);
  // Warps to a token's queries: as many as keep a lane one batch busy while the SMs have room for 32 warps each.
  const int64_t items = (int64_t)Hq * (D * bytes / 32);
  w.share = 1;
  while (w.share < 16 && (int64_t)T * w.share < 32LL * sms && (int64_t)w.share * 32 < items) w.share *= 2;
  w.query_ctas = Hq > 0 ? ((int64_t)T * w.share + kWarps - 1) / kWarps : 0;
  // Queries' CTAs wait for memory and groups' for their steps: where not all fit at once they take turns (8000 tokens 41.3 us
  // with the groups' first, 37.6 in turn; 100 tokens 5.7 and 6.1).
  w.turns = w.group_ctas + w.query_ctas > at_once ? std::min(w.group_ctas, w.query_ctas) : 0;
  w.rows = rows_of_round(w.heads_of, D, bytes);
  const size_t sines = rotate ? (size_t)D * sizeof(float) : 0;
  w.smem = std::max(w.rows * (2 * w.heads_of * ((size_t)D * bytes + sizeof(float)) + sines), kWarps * sines);
  return w;
}

}  // namespace scaled
}  // namespace isk
