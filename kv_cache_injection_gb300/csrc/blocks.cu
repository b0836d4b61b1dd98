// Block tables and slot maps of a step's new tokens (is_extend_block_table).
//
// With n tokens in the cache and m new ones, a request holds ceil(n / bs)
// blocks and needs ceil((n + m) / bs); its missing blocks are the free-list
// entries from *head + (blocks missing before it) on, its packed tokens start
// at the sum of the new lengths before it, and token i's slot is
// block[(n + i) / bs] * bs + (n + i) % bs.  Both sums are prefix sums over at
// most IS_MAX_REQUESTS requests, 32 KB of input: every CTA computes them for
// itself instead of waiting for another, so the call is one launch and no CTA
// depends on what another writes (a new token's block id comes from the free
// list, not from the table entry).  Bound by latency at few tokens (100
// requests of one token: 3.6 us) and by the instructions of going over all
// requests in every CTA at many (4096 requests, 614,000 tokens, 7.7 MB: 8.6
// us; 45 with 64-bit divisions and a search per token).
#include <algorithm>

#include "block_scan.cuh"
#include "common.cuh"
#include "internal.h"

namespace isk {

// Few requests: small CTAs, one token and at most two requests a thread.  Many:
// large ones, since each CTA goes over all requests (4096 requests: 11.5 us
// with 512 threads a CTA, 8.6 with 1024).
constexpr int kFewRequests = 512, kFewThreads = 256, kManyThreads = 1024;
constexpr int kFewTokens = 1, kManyTokens = 4;   // tokens a thread

// Division by the block size as a multiplication: with 2^(k-1) < bs <= 2^k and
// mul = ceil(2^(26+k) / bs), x / bs = x * mul >> (26 + k) for every x < 2^26
// (mul overshoots 2^(26+k) / bs by less than 1, so x * mul / 2^(26+k) by less
// than 2^-k <= 1 / bs, which carries no quotient over the next whole number).
// Lengths stay below 2^24 + 1 and block sizes at most 2^24, so x < 2^26.
struct BlockDiv {
  uint32_t mul, shift;
};
static BlockDiv block_div(int32_t bs) {
  uint32_t k = 0;
  while ((1ll << k) < bs) ++k;
  return {(uint32_t)(((1ull << (26 + k)) + (uint64_t)bs - 1) / (uint64_t)bs), 26 + k};
}
__device__ __forceinline__ int32_t div_bs(int32_t x, const BlockDiv& d) {
  return (int32_t)(((uint64_t)(uint32_t)x * d.mul) >> d.shift);
}
__device__ __forceinline__ int32_t blocks_of(int32_t n, int32_t bs, const BlockDiv& d) { return div_bs(n + bs - 1, d); }

// Request r's place in the shared tables: threads that walk 2 or 4 consecutive
// requests each then hit different banks.
__host__ __device__ constexpr int at(int r) { return r + (r >> 5); }

template <int kExtendThreads, int kPer, int kTokensPerThread>
__global__ void __launch_bounds__(kExtendThreads) extend_kernel(const is_extend_args_t a, const BlockDiv div) {
  extern __shared__ int32_t sm[];
  __shared__ int64_t scratch[2][33];
  __shared__ int32_t s_used;
  const int R = a.num_requests, bs = a.block_size, tid = threadIdx.x;
  const int pitch = at(R) + 1;
  int32_t* s_start = sm;                 // [R + 1] first packed token, INT32_MAX at most
  int32_t* s_seq = sm + pitch;           // [R] seq_len, or -1 if the request is refused
  int32_t* s_taken = s_seq + pitch;      // [R] blocks taken before the request (what matters of it is at most num_free)
  pdl_wait();
  pdl_trigger();
  int32_t head = a.free_head ? a.free_head[0] : 0;
  uint32_t bits = 0;
  if (head < 0 || head > a.num_free) {
    bits |= IS_ST_FREE_LIST;
    head = a.num_free;
  }
  const int32_t avail = a.num_free - head;
  if (tid == 0) s_used = 0;
  constexpr int kTokensPerCta = kExtendThreads * kTokensPerThread;
  // A thread's requests are consecutive; all their lengths are loaded before any is used.
  const int r0 = min(R, tid * kPer), r1 = min(R, r0 + kPer);
  int32_t len[kPer], add[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const bool in = r0 + i < r1;
    len[i] = in ? a.seq_len[r0 + i] : 0;
    add[i] = in ? a.new_len[r0 + i] : 0;
  }
  int32_t lack[kPer];                    // blocks missing
  int64_t tokens = 0, missing = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (r0 + i >= r1) continue;
    const int32_t n = len[i], m = add[i];
    add[i] = min(max(m, 0), IS_MAX_POSITION);
    int32_t miss = 0;
    if (n < 0 || m < 0) {
      bits |= IS_ST_COUNT;
      len[i] = -1;
    } else if ((int64_t)n + m > IS_MAX_POSITION) {
      bits |= IS_ST_POSITION;
      len[i] = -1;
    } else {
      const int32_t need = blocks_of(n + m, bs, div);
      if (m > 0 && need > a.max_blocks_per_seq) {
        bits |= IS_ST_BLOCK_TABLE;
        len[i] = -1;
      } else {
        miss = need - blocks_of(n, bs, div);
      }
    }
    lack[i] = miss;
    tokens += add[i];
    missing += miss;
  }
  int64_t total, all_missing;
  // One barrier a sum while adding up the warps' totals is cheap, three with many warps.
  auto scan = [](int64_t x, int64_t* scratch_, int64_t* sum) {
    if constexpr (kExtendThreads <= 256) return block_exclusive_scan_1bar<kExtendThreads / 32>(x, scratch_, sum);
    else return block_exclusive_scan(x, scratch_, sum);
  };
  int64_t first = scan(tokens, scratch[0], &total);
  int64_t taken = scan(missing, scratch[1], &all_missing);
  int32_t used = 0;                      // blocks taken up to this thread's last request
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int r = r0 + i;
    if (r >= r1) continue;
    const int32_t miss = lack[i];
    s_start[at(r)] = (int32_t)min(first, (int64_t)INT32_MAX);
    if (len[i] >= 0 && miss > 0) {
      if (taken + miss > avail) {
        bits |= IS_ST_FREE_LIST;
        len[i] = -1;
      } else {
        used = (int32_t)(taken + miss);
      }
    }
    s_seq[at(r)] = len[i];
    s_taken[at(r)] = (int32_t)min(taken, (int64_t)INT32_MAX);
    first += add[i];
    taken += miss;
  }
  used = __reduce_max_sync(0xffffffffu, used);
  if ((tid & 31) == 0) atomicMax(&s_used, used);
  if (tid == 0) s_start[at(R)] = (int32_t)min(total, (int64_t)INT32_MAX);
  if (total > a.max_tokens) bits |= IS_ST_COUNT;
  __syncthreads();

  // Slots and positions of this CTA's packed tokens.  A warp has consecutive ones and finds the requests of its first
  // and last together, 32 probes at a time; each lane's request lies between the two.  All block ids are loaded before
  // any is used.
  const int lane = tid & 31;
  const int32_t end = s_start[at(R)];
  const int64_t tw = (int64_t)blockIdx.x * kTokensPerCta + (int64_t)(tid >> 5) * 32 * kTokensPerThread;   // the warp's first
  auto find_warp = [&](int32_t t) {      // last request that starts at or before t
    int lo = 0, hi = R;
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) >> 5, idx = lo + lane * step;
      const unsigned m = __ballot_sync(0xffffffffu, idx < hi && s_start[at(idx)] <= t);   // lane 0 probes lo, which qualifies
      lo += (31 - __clz(m)) * step;
      hi = min(hi, lo + step);
    }
    return lo;
  };
  int32_t pos[kTokensPerThread], id[kTokensPerThread];
  const int32_t t_last = (int32_t)min(min((int64_t)end, (int64_t)a.max_tokens) - 1, tw + 32 * kTokensPerThread - 1);
  const int r_first = tw <= t_last ? find_warp((int32_t)tw) : 0, r_last = tw <= t_last ? find_warp(t_last) : 0;
#pragma unroll
  for (int i = 0; i < kTokensPerThread; ++i) {
    const int64_t t64 = tw + i * 32 + lane;
    pos[i] = -1;
    id[i] = -1;
    if (t64 > t_last) continue;
    const int32_t t = (int32_t)t64;
    int lo = r_first, hi = r_last + 1;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_start[at(mid)] <= t) lo = mid; else hi = mid;
    }
    const int32_t n = s_seq[at(lo)];
    if (n < 0) continue;
    pos[i] = n + (t - s_start[at(lo)]);
    const int32_t j = div_bs(pos[i], div);
    const int32_t have = blocks_of(n, bs, div);
    const int32_t* src = j >= have ? a.free_blocks + (head + s_taken[at(lo)] + (j - have))
                                   : a.block_table + ((size_t)lo * a.max_blocks_per_seq + j);
    id[i] = *src;
  }
#pragma unroll
  for (int i = 0; i < kTokensPerThread; ++i) {
    const int64_t t = tw + i * 32 + lane;
    if (t >= a.max_tokens) continue;
    int64_t slot = -1;
    if (pos[i] >= 0) {
      if (id[i] < 0 || id[i] >= a.num_blocks)
        bits |= IS_ST_BLOCK_ID;
      else
        slot = (int64_t)id[i] * bs + (pos[i] - div_bs(pos[i], div) * bs);
    }
    a.slot_mapping_out[t] = slot;
    if (t < end && a.positions_out) a.positions_out[t] = pos[i];
  }

  // Table entries: the blocks taken are the free list's next s_used, one thread each.  (64-bit steps: slot maps of
  // almost 2^31 entries have 2^31 threads.)
  const int32_t all_used = s_used;
  const int64_t threads = (int64_t)gridDim.x * kExtendThreads, me = (int64_t)blockIdx.x * kExtendThreads + tid;
  for (int64_t i64 = me; i64 < all_used; i64 += threads) {
    const int32_t i = (int32_t)i64;
    int lo = 0, hi = R;                  // last request with at most i blocks taken before it: the one that takes block i
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_taken[at(mid)] <= i) lo = mid; else hi = mid;
    }
    a.block_table[(size_t)lo * a.max_blocks_per_seq + blocks_of(s_seq[at(lo)], bs, div) + (i - s_taken[at(lo)])] =
        a.free_blocks[head + i];
  }
  // Per-request outputs.
  for (int64_t r64 = me; r64 < R; r64 += threads) {
    const int r = (int)r64;
    const int32_t n = s_seq[at(r)];
    if (a.seq_len_out) a.seq_len_out[r] = n >= 0 ? n + a.new_len[r] : a.seq_len[r];
    if (a.token_start_out) {
      a.token_start_out[r] = s_start[at(r)];
      if (r == R - 1) a.token_start_out[R] = end;
    }
  }
  if (blockIdx.x == 0 && tid == 0 && a.free_head_out) a.free_head_out[0] = head + s_used;
  if (bits) latch(a.status_out, bits);
}

template <int THREADS, int PER, int TOKENS>
static cudaError_t launch_extend_t(const is_extend_args_t& a, const LaunchCfg& cfg) {
  auto* kern = extend_kernel<THREADS, PER, TOKENS>;
  const size_t smem = (size_t)3 * (at(a.num_requests) + 1) * sizeof(int32_t);
  const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  constexpr int per_cta = THREADS * TOKENS;
  const int grid = (int)(((int64_t)a.max_tokens + per_cta - 1) / per_cta);
  return launch_ex(kern, dim3(grid), dim3(THREADS), smem, cfg.stream, cfg.pdl, a, block_div(a.block_size));
}

cudaError_t launch_extend(const is_extend_args_t& a, const LaunchCfg& cfg) {
  static_assert(kFewRequests <= kFewThreads * 2 && IS_MAX_REQUESTS <= kManyThreads * 4, "every request has a thread");
  return a.num_requests <= kFewRequests ? launch_extend_t<kFewThreads, 2, kFewTokens>(a, cfg)
                                        : launch_extend_t<kManyThreads, 4, kManyTokens>(a, cfg);
}

}  // namespace isk
