// How a write into a scaled cache is spread over CTAs (scaled.cu).  Host code
// without CUDA, so that it is tested as it is.
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>

namespace isk {
namespace scaled {

// 128 threads and 32 KB of rows, three to six CTAs an SM: the steps of a CTA wait for one another, other CTAs fill the gaps
// (8000 tokens 37 us, 51 with 256 threads and 64 KB, 45 with 128 threads and 16 KB).
constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kWindow = 30;              // tokens of a CTA, at most (a warp looks at them and a neighbour)
constexpr int kMaxGroups = 16;           // of a round
constexpr int kMaxRows = 128;            // of a round
constexpr int kDataBytes = 32768;        // of a round's rows: keys and values of the CTA's heads
constexpr int kMaxUnits = 8;             // a head's keys, or its values

// Rows of a round of a CTA with `heads_of` heads.
inline int rows_of_round(int heads_of, int D, int bytes) { return std::min(kMaxRows, kDataBytes / (2 * heads_of * D * bytes)); }

// Bytes of shared memory that a launch asks for: a round's rows, a largest element for each of their units, their keys'
// sines; or a row of sines for each warp of a queries' CTA.
inline size_t smem_of(int heads_of, int D, int bytes, bool rotate) {
  const size_t sines = rotate ? (size_t)D * sizeof(float) : 0;
  return std::max(rows_of_round(heads_of, D, bytes) * (2 * heads_of * ((size_t)D * bytes + sizeof(float)) + sines), kWarps * sines);
}

// CTAs that an SM holds: as many as its registers do (the launch bounds), if their shared memory, 3 KB of it static and 1 KB
// the system's, fits 228 KB.  With keys of head_dim 128 in 16 bits to rotate five of four heads, four of two, three of one.
constexpr int most_per_sm(bool rotate) { return rotate ? 5 : 6; }
inline int per_sm(int heads_of, int D, int bytes, bool rotate) {
  return std::min(most_per_sm(rotate), (int)(228 * 1024 / (smem_of(heads_of, D, bytes, rotate) + 4096)));
}

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
  // Warps to a token's queries: as many as keep a lane one batch busy while the SMs have room for 32 warps each.
  const int64_t items = (int64_t)Hq * (D * bytes / 32);
  w.share = 1;
  while (w.share < 16 && (int64_t)T * w.share < 32LL * sms && (int64_t)w.share * 32 < items) w.share *= 2;
  w.query_ctas = Hq > 0 ? ((int64_t)T * w.share + kWarps - 1) / kWarps : 0;
  // Two heads too where the CTAs then fit at once: one token 5.5 -> 5.0 us, 1276 moved tokens 7.6 -> 6.6.  Of an append the
  // queries' CTAs count too; where they come to more than five an SM in all, as with all but the shortest prompts, the groups'
  // may take two thirds of the places (32 + 8 heads, two and four: 120 single tokens 5.4 and 6.2 us, 160 9.0 and 6.6, 1000
  // 15.6 and 10.8, a prompt of 2400 18.1 and 14.5; 28 + 4 heads: 456 single tokens 6.4 and 7.4, 300 9.4 and 6.4, a prompt of
  // 1276 9.4 and 10.7, of 6000 24.8 and 21.6).
  const int64_t windows = ((int64_t)T + w.window - 1) / w.window, five = 5LL * sms;
  auto groups_of = [&](int heads_of) { return windows * ((H + heads_of - 1) / heads_of); };
  auto places_of = [&](int heads_of) { return (int64_t)sms * per_sm(heads_of, D, bytes, rotate); };
  if (w.heads_of > 2) {
    const bool many = w.query_ctas > 0 && groups_of(2) + w.query_ctas > five;
    if (groups_of(2) <= (many ? places_of(2) * 2 / 3 : places_of(2))) w.heads_of = 2;
  }
  // One head where two heads' rows of a block do not fit a round, CTAs have several tokens and are at most ten an SM (a move's
  // twelve), most of which have no group then: into blocks of 64, 1276 moved tokens 9.7 us, 15.0 with two, 6000 14.0 and 19.5,
  // 8000 19.5 and 21.4; a prompt of 1276 23.2 and 30.3, of 8000 65 and 55.  (305 to 2000 single tokens, which cannot be told
  // from a prompt here, lose by it: 1000 take 26 us, not 16.)
  if (w.heads_of == 2 && w.window > 1 && groups_of(1) <= 2LL * sms * most_per_sm(rotate) &&
      rows_of_round(2, D, bytes) < std::min(block_size, kMaxRows))
    w.heads_of = 1;
  w.group_ctas = groups_of(w.heads_of);
  // Queries' CTAs wait for memory and groups' for their steps: from five an SM on they take turns (8000 tokens 41.3 us with
  // the groups' first, 37.6 in turn; 100 tokens 5.7 and 6.1).
  w.turns = w.group_ctas + w.query_ctas > five ? std::min(w.group_ctas, w.query_ctas) : 0;
  w.rows = rows_of_round(w.heads_of, D, bytes);
  w.smem = smem_of(w.heads_of, D, bytes, rotate);
  return w;
}

}  // namespace scaled
}  // namespace isk
