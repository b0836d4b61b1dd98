// C ABI of the serving step around the segment: argument checks and launches of
// is_extend_block_table, is_append and is_attend.  They keep no state but a
// thread's last rotation table, which its parameters determine (axis_turns): the
// device comes from the call's buffers, everything else from its arguments.
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <mutex>

#include "common.cuh"
#include "internal.h"

using namespace isk;

namespace {

is_status_t refuse(is_status_t s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  set_last_error_message(buf);
  return s;
}

is_status_t launched(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return IS_OK;
  cudaGetLastError();                    // reported here, not again by a later call
  return refuse(IS_ERR_CUDA, "%s failed: %s", what, cudaGetErrorString(e));
}

// Device that owns `p`, which must be device or managed memory.
is_status_t device_of(const void* p, const char* name, int* dev) {
  cudaPointerAttributes at;
  const cudaError_t e = cudaPointerGetAttributes(&at, p);
  if (e != cudaSuccess) return launched(e, "cudaPointerGetAttributes");
  if (at.type == cudaMemoryTypeManaged) return launched(cudaGetDevice(dev), "cudaGetDevice");
  if (at.type != cudaMemoryTypeDevice) return refuse(IS_ERR_INVALID_ARG, "%s is not device memory", name);
  *dev = at.device;
  return IS_OK;
}

int sms_of(int dev) {
  static std::mutex mu;
  static int sms[64];
  if (dev < 0 || dev >= 64) return 0;
  std::lock_guard<std::mutex> lock(mu);
  if (sms[dev] == 0 && cudaDeviceGetAttribute(&sms[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    sms[dev] = 0;
  }
  return sms[dev];
}

struct Span {
  const char* name;
  uintptr_t lo, hi;
  Span(const char* n, const void* p, int64_t bytes)
      : name(n), lo((uintptr_t)p), hi(p ? (uintptr_t)p + (uintptr_t)bytes : (uintptr_t)p) {}
  bool meets(const Span& o) const { return lo < o.hi && o.lo < hi; }
};

// No output may share a byte with an input or with another output.
is_status_t check_apart(const Span* outs, int n_out, const Span* ins, int n_in) {
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < n_in; ++j)
      if (outs[i].meets(ins[j])) return refuse(IS_ERR_INVALID_ARG, "%s overlaps %s", outs[i].name, ins[j].name);
    for (int j = i + 1; j < n_out; ++j)
      if (outs[i].meets(outs[j])) return refuse(IS_ERR_INVALID_ARG, "%s overlaps %s", outs[i].name, outs[j].name);
  }
  return IS_OK;
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

is_status_t check_layer_cache(const is_cache_desc_t& c, int dtype, const void* layer_cache) {
  if (c.block_size < 1 || c.block_size > IS_MAX_POSITION || c.num_blocks < 1)
    return refuse(IS_ERR_INVALID_ARG, "block_size must be in [1, IS_MAX_POSITION], num_blocks >= 1");
  if (c.dtype == IS_FP8_E4M3) {
    if (dtype == IS_F32) return refuse(IS_ERR_UNSUPPORTED, "an FP8 cache goes with bf16 or fp16");
    if (!(c.k_scale > 0.f) || !(c.v_scale > 0.f) || !std::isfinite(c.k_scale) || !std::isfinite(c.v_scale))
      return refuse(IS_ERR_INVALID_ARG, "FP8 cache scales must be finite and > 0");
  } else if (c.dtype != dtype) {
    return refuse(IS_ERR_INVALID_ARG, "cache dtype %d differs from the call's dtype %d", c.dtype, dtype);
  }
  if (!aligned16(layer_cache)) return refuse(IS_ERR_INVALID_ARG, "layer_cache must be 16-byte aligned");
  return IS_OK;
}

bool valid_dtype(int dt) { return dt == IS_F32 || dt == IS_BF16 || dt == IS_F16; }

// The rotation turns of (rope, axes, D).  A step calls is_append once per layer
// with the same parameters, so the calling thread keeps the last ones by value.
is_status_t axis_turns(const is_rope_params_t& r, const is_rope_axes_t& x, int D, const AxisTurns** out) {
  struct Kept {
    bool valid = false;
    is_rope_params_t r;
    is_rope_axes_t x;
    int D;
    AxisTurns t;
  };
  static thread_local Kept kept;
  const int half = D / 2;
  if (kept.valid && kept.D == D && std::memcmp(&kept.x, &x, sizeof x) == 0 &&
      std::memcmp(&kept.r, &r, offsetof(is_rope_params_t, original_max_pos) + 4) == 0) {
    *out = &kept.t;
    return IS_OK;
  }
  if (x.reserved != 0) return refuse(IS_ERR_INVALID_ARG, "axes.reserved must be 0");
  if (x.n_axes < 1 || x.n_axes > IS_MAX_ROPE_AXES)
    return refuse(IS_ERR_INVALID_ARG, "n_axes must be in [1, IS_MAX_ROPE_AXES]");
  if (x.interleaved != 0 && x.interleaved != 1) return refuse(IS_ERR_INVALID_ARG, "axes.interleaved must be 0 or 1");
  kept.valid = false;
  std::memset(&kept.t, 0, sizeof kept.t);
  if (x.n_axes > 1) {
    int64_t sum = 0;
    for (int a = 0; a < x.n_axes; ++a) {
      if (x.section[a] < 0) return refuse(IS_ERR_INVALID_ARG, "a section is negative");
      sum += x.section[a];
    }
    if (sum != half) return refuse(IS_ERR_INVALID_ARG, "the sections must add up to head_dim / 2");
    if (x.interleaved) {
      for (int a = 1; a < x.n_axes; ++a)
        for (int j = 0; j < x.section[a]; ++j) {
          const int i = a + j * x.n_axes;
          if (i >= half) return refuse(IS_ERR_INVALID_ARG, "interleaved section %d does not fit the head", a);
          kept.t.axis[i] = (uint8_t)a;
        }
    } else {
      for (int a = 0, i = 0; a < x.n_axes; ++a)
        for (int j = 0; j < x.section[a]; ++j) kept.t.axis[i++] = (uint8_t)a;
    }
  }
  double w[kMaxHalfDim];
  const is_status_t st = is_rope_frequencies(&r, D, w);
  if (st != IS_OK) return st;
  for (int i = 0; i < half; ++i) {
    const double turns = w[i] / 6.283185307179586476925286766559;
    kept.t.t.hi[i] = (float)turns;
    kept.t.t.lo[i] = (float)(turns - (double)kept.t.t.hi[i]);
  }
  kept.r = r;
  kept.x = x;
  kept.D = D;
  kept.valid = true;
  *out = &kept.t;
  return IS_OK;
}

}  // namespace

extern "C" is_status_t is_extend_block_table(const is_extend_args_t* a, cudaStream_t stream) {
  if (!a) return refuse(IS_ERR_INVALID_ARG, "args are NULL");
  if (!a->seq_len || !a->new_len || !a->block_table || !a->slot_mapping_out || !a->status_out ||
      (!a->free_blocks && a->num_free > 0))
    return refuse(IS_ERR_INVALID_ARG, "a required pointer is NULL");
  if (a->num_requests < 1 || a->num_requests > IS_MAX_REQUESTS)
    return refuse(IS_ERR_INVALID_ARG, "num_requests must be in [1, IS_MAX_REQUESTS]");
  if (a->num_free < 0 || a->block_size < 1 || a->block_size > IS_MAX_POSITION || a->num_blocks < 1 ||
      a->max_blocks_per_seq < 1 || a->max_tokens < 1)
    return refuse(IS_ERR_INVALID_ARG,
                  "num_free must be >= 0, block_size in [1, IS_MAX_POSITION]; num_blocks, max_blocks_per_seq, "
                  "max_tokens >= 1");
  const int64_t R = a->num_requests;
  const Span ins[] = {{"seq_len", a->seq_len, 4 * R}, {"new_len", a->new_len, 4 * R},
                      {"free_blocks", a->free_blocks, 4LL * a->num_free}, {"free_head", a->free_head, 4}};
  const Span outs[] = {{"block_table", a->block_table, 4LL * R * a->max_blocks_per_seq},
                       {"slot_mapping_out", a->slot_mapping_out, 8LL * a->max_tokens},
                       {"positions_out", a->positions_out, 4LL * a->max_tokens},
                       {"token_start_out", a->token_start_out, 4 * (R + 1)},
                       {"seq_len_out", a->seq_len_out, 4 * R},
                       {"free_head_out", a->free_head_out, 4},
                       {"status_out", a->status_out, 4}};
  is_status_t st = check_apart(outs, 7, ins, 4);
  if (st != IS_OK) return st;
  int dev = 0;
  st = device_of(a->slot_mapping_out, "slot_mapping_out", &dev);
  if (st != IS_OK) return st;
  DeviceGuard g(dev);
  return launched(launch_extend(*a, LaunchCfg{stream, sms_of(dev), true}), "is_extend_block_table launch");
}

extern "C" is_status_t is_append(const is_append_args_t* a, cudaStream_t stream) {
  if (!a) return refuse(IS_ERR_INVALID_ARG, "args are NULL");
  const int T = a->num_tokens, Hq = a->num_q_heads, H = a->num_kv_heads, D = a->head_dim;
  if (T < 0 || Hq < 0 || H < 1) return refuse(IS_ERR_INVALID_ARG, "num_tokens, num_q_heads >= 0, num_kv_heads >= 1");
  if (!valid_dtype(a->dtype)) return refuse(IS_ERR_INVALID_ARG, "bad dtype");
  if (a->reserved != 0 || a->reserved2 != 0) return refuse(IS_ERR_INVALID_ARG, "reserved must be 0");
  if (D < 16 || D > IS_MAX_HEAD_DIM || (D & (D - 1)) != 0)
    return refuse(IS_ERR_UNSUPPORTED, "head_dim must be a power of two in [16, IS_MAX_HEAD_DIM]");
  if (Hq > (1 << 16) || H > (1 << 16)) return refuse(IS_ERR_UNSUPPORTED, "at most 65536 heads");
  is_status_t st = check_layer_cache(a->cache, a->dtype, a->layer_cache);
  if (st != IS_OK) return st;
  const int e = a->dtype == IS_F32 ? 4 : 2, ve = 16 / e;
  const AxisTurns* turns = nullptr;
  st = axis_turns(a->rope, a->axes, D, &turns);
  if (st != IS_OK) return st;
  const int vecs = a->rope.style == 0 ? D / 2 / ve : D / ve;
  if (vecs < 1 || vecs > 32)
    return refuse(IS_ERR_UNSUPPORTED, "head_dim %d with this dtype/style needs %d vectors per %s", D, vecs,
                  a->rope.style == 0 ? "half head (max 32)" : "head (max 32)");
  if (T == 0) return IS_OK;
  if (!a->k || !a->v || !a->positions || !a->slot_mapping || !a->layer_cache || !a->status_out ||
      (Hq > 0 && (!a->q || !a->q_out)))
    return refuse(IS_ERR_INVALID_ARG, "a required pointer is NULL");
  const int64_t qrow = (int64_t)Hq * D, row = (int64_t)H * D;
  if ((Hq > 0 && T > 1 && a->q_stride < qrow) || (T > 1 && (a->k_stride < row || a->v_stride < row)))
    return refuse(IS_ERR_INVALID_ARG, "a stride is smaller than its row");
  const int64_t qs = Hq > 0 ? a->q_stride * e : 0, ks = a->k_stride * e, vs = a->v_stride * e;
  if ((T > 1 && ((qs | ks | vs) & 15)) || !aligned16(a->k) || !aligned16(a->v) ||
      (Hq > 0 && (!aligned16(a->q) || !aligned16(a->q_out))))
    return refuse(IS_ERR_INVALID_ARG, "rows of q, k, v and q_out must be 16-byte aligned");
  const int c = a->cache.dtype == IS_FP8_E4M3 ? 1 : e;
  const int64_t slots = (int64_t)a->cache.num_blocks * a->cache.block_size;
  const Span sq("q", Hq > 0 ? a->q : nullptr, (T - 1) * qs + qrow * e);
  const Span ins[] = {{"k", a->k, (T - 1) * ks + row * e}, {"v", a->v, (T - 1) * vs + row * e},
                      {"positions", a->positions, 4LL * T * a->axes.n_axes}, {"slot_mapping", a->slot_mapping, 8LL * T},
                      sq};
  const Span outs[] = {{"layer_cache", a->layer_cache, 2 * slots * row * c}, {"status_out", a->status_out, 4},
                       {"q_out", Hq > 0 ? a->q_out : nullptr, T * qrow * e}};
  const bool in_place = Hq > 0 && a->q == a->q_out && (T == 1 || a->q_stride == qrow);
  st = check_apart(outs, 2, ins, 5);
  if (st == IS_OK) st = check_apart(outs + 2, 1, ins, in_place ? 4 : 5);
  if (st == IS_OK) st = check_apart(outs, 3, nullptr, 0);
  if (st != IS_OK) return st;
  int dev = 0;
  st = device_of(a->layer_cache, "layer_cache", &dev);
  if (st != IS_OK) return st;

  AppendArgs p{};
  p.q = static_cast<const uint8_t*>(a->q);
  p.k = static_cast<const uint8_t*>(a->k);
  p.v = static_cast<const uint8_t*>(a->v);
  p.q_stride = qs;
  p.k_stride = ks;
  p.v_stride = vs;
  p.positions = a->positions;
  p.slots = a->slot_mapping;
  p.q_out = static_cast<uint8_t*>(a->q_out);
  p.k_cache = static_cast<uint8_t*>(a->layer_cache);
  p.v_offset = slots * row * c;
  p.n_slots = slots;
  p.status = a->status_out;
  p.T = T;
  p.Hq = Hq;
  p.H = H;
  p.D = D;
  p.n_axes = a->axes.n_axes;
  p.dtype = a->dtype;
  p.style = a->rope.style;
  p.fp8 = a->cache.dtype == IS_FP8_E4M3;
  if (p.fp8) {
    p.k_inv = (float)(1.0 / (double)a->cache.k_scale);
    p.v_inv = (float)(1.0 / (double)a->cache.v_scale);
  }
  DeviceGuard g(dev);
  return launched(launch_append(p, *turns, LaunchCfg{stream, sms_of(dev), true}), "is_append launch");
}

extern "C" is_status_t is_attend(const is_attend_args_t* args, cudaStream_t stream) {
  return is_attend_within(args, (int64_t)kWaitBudgetNs, stream);
}

extern "C" is_status_t is_attend_within(const is_attend_args_t* a, int64_t budget_ns, cudaStream_t stream) {
  if (!a) return refuse(IS_ERR_INVALID_ARG, "args are NULL");
  if (budget_ns < 0 || budget_ns > (int64_t)kWaitBudgetNs)
    return refuse(IS_ERR_INVALID_ARG, "budget_ns must be in [0, %llu]", (unsigned long long)kWaitBudgetNs);
  const int R = a->num_requests, T = a->num_tokens, Hq = a->num_q_heads, H = a->num_kv_heads, D = a->head_dim;
  if (R < 1 || R > IS_MAX_REQUESTS) return refuse(IS_ERR_INVALID_ARG, "num_requests must be in [1, IS_MAX_REQUESTS]");
  if (T < 0 || a->max_q_len < 1 || a->max_blocks_per_seq < 1 || a->window < 0)
    return refuse(IS_ERR_INVALID_ARG, "num_tokens, window >= 0; max_q_len, max_blocks_per_seq >= 1");
  if (H < 1 || Hq < 1 || Hq % H != 0)
    return refuse(IS_ERR_INVALID_ARG, "num_q_heads must be a positive multiple of num_kv_heads");
  if (!valid_dtype(a->dtype)) return refuse(IS_ERR_INVALID_ARG, "bad dtype");
  if (a->reserved != 0) return refuse(IS_ERR_INVALID_ARG, "reserved must be 0");
  if (!std::isfinite(a->scale)) return refuse(IS_ERR_INVALID_ARG, "scale must be finite");
  if (D != 64 && D != 128 && D != 256) return refuse(IS_ERR_UNSUPPORTED, "head_dim must be 64, 128 or 256");
  if (Hq > (1 << 16) || (int64_t)T * Hq > (1 << 30))
    return refuse(IS_ERR_UNSUPPORTED, "at most 65536 heads and 2^30 rows (num_tokens * num_q_heads)");
  is_status_t st = check_layer_cache(a->cache, a->dtype, a->layer_cache);
  if (st != IS_OK) return st;
  if (!a->q_start && T < R) return refuse(IS_ERR_INVALID_ARG, "without q_start there is one row per request");
  if (T == 0) return IS_OK;
  if (!a->q || !a->seq_len || !a->block_table || !a->layer_cache || !a->out || !a->workspace || !a->status_out)
    return refuse(IS_ERR_INVALID_ARG, "a required pointer is NULL");
  if (a->workspace_bytes < IS_ATTEND_WORKSPACE_BYTES)
    return refuse(IS_ERR_INVALID_ARG, "workspace must hold IS_ATTEND_WORKSPACE_BYTES");
  const int e = a->dtype == IS_F32 ? 4 : 2;
  const int64_t qrow = (int64_t)Hq * D, row = (int64_t)H * D;
  if (T > 1 && a->q_stride < qrow) return refuse(IS_ERR_INVALID_ARG, "q_stride is smaller than a row");
  const int64_t qs = a->q_stride * e;
  if ((T > 1 && (qs & 15)) || !aligned16(a->q))
    return refuse(IS_ERR_INVALID_ARG, "rows of q must be 16-byte aligned");
  if (((uintptr_t)a->out | (uintptr_t)a->workspace) & 31)
    return refuse(IS_ERR_INVALID_ARG, "out and workspace must be 32-byte aligned");
  const int c = a->cache.dtype == IS_FP8_E4M3 ? 1 : e;
  const int64_t slots = (int64_t)a->cache.num_blocks * a->cache.block_size;
  const Span ins[] = {{"q", a->q, (T - 1) * qs + qrow * e}, {"q_start", a->q_start, 4LL * (R + 1)},
                      {"seq_len", a->seq_len, 4LL * R}, {"block_table", a->block_table, 4LL * R * a->max_blocks_per_seq},
                      {"layer_cache", a->layer_cache, 2 * slots * row * c}};
  const Span outs[] = {{"out", a->out, T * qrow * e}, {"lse_out", a->lse_out, 4LL * T * Hq},
                       {"workspace", a->workspace, IS_ATTEND_WORKSPACE_BYTES}, {"status_out", a->status_out, 4}};
  st = check_apart(outs, 4, ins, 5);
  if (st != IS_OK) return st;
  int dev = 0;
  st = device_of(a->out, "out", &dev);
  if (st != IS_OK) return st;

  AttendArgs p{};
  p.q = static_cast<const uint8_t*>(a->q);
  p.q_stride = qs;
  p.q_start = a->q_start;
  p.seq_len = a->seq_len;
  p.block_table = a->block_table;
  p.k_cache = static_cast<const uint8_t*>(a->layer_cache);
  p.v_offset = slots * row * c;
  p.out = static_cast<uint8_t*>(a->out);
  p.lse = a->lse_out;
  p.workspace = static_cast<uint8_t*>(a->workspace);
  p.status = a->status_out;
  p.R = R;
  p.T = T;
  p.max_q = a->q_start ? a->max_q_len : 1;
  if (p.max_q > T) p.max_q = T;          // more rows than T are out of range in any case
  p.Hq = Hq;
  p.H = H;
  p.G = Hq / H;
  p.D = D;
  p.max_blocks = a->max_blocks_per_seq;
  p.block_size = a->cache.block_size;
  p.num_blocks = a->cache.num_blocks;
  p.block_shift = -1;
  for (int s = 0; s <= 24; ++s)
    if (a->cache.block_size == 1 << s) p.block_shift = s;
  p.window = a->window;
  p.dtype = a->dtype;
  p.fp8 = a->cache.dtype == IS_FP8_E4M3;
  p.scale = p.fp8 ? a->scale * a->cache.k_scale : a->scale;
  p.v_scale = p.fp8 ? a->cache.v_scale : 1.f;
  p.wait_ns = (uint64_t)budget_ns;
  DeviceGuard g(dev);
  return launched(launch_attend(p, LaunchCfg{stream, sms_of(dev), true}), "is_attend launch");
}
