// Entry points of the rotary positions, the 8-bit key/value cache and the
// attention over it: argument checks and status codes. Nothing here computes
// on the host but mq_rope_table.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "../../include/mq.h"
#include "kv_internal.h"
#include "mq_device.cuh"
#include "mq_internal.h"

namespace mq {
namespace {

mq_status refuse(mq_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  set_last_error(buf);
  return s;
}

mq_status finish(cudaError_t e, const char* who) {
  if (e == cudaSuccess) return MQ_OK;
  if (e == cudaErrorNotSupported) return refuse(MQ_ERR_UNSUPPORTED, "%s: sizes not served by this build", who);
  return refuse(MQ_ERR_CUDA, "%s: %s", who, cudaGetErrorString(e));
}

bool on(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool is_dtype(int d) { return d == MQ_F32 || d == MQ_BF16; }

mq_status check_rope(const char* who, const mq_rope_positions* r, int64_t d, int unit, Rope* out) {
  if (!r->turns || !on(r->turns, 8)) return refuse(MQ_ERR_INVALID_ARG, "%s: rope turns null or not 8-byte aligned", who);
  if (r->rot_dim < 2 || r->rot_dim > d || r->rot_dim % 2 != 0)
    return refuse(MQ_ERR_INVALID_ARG, "%s: rot_dim=%d must be even and in [2, head_dim]", who, r->rot_dim);
  if (r->rot_dim % unit != 0)
    return refuse(MQ_ERR_UNSUPPORTED, "%s: rot_dim=%d must be a multiple of %d here", who, r->rot_dim, unit);
  if (r->layout != MQ_ROPE_HALF && r->layout != MQ_ROPE_INTERLEAVED)
    return refuse(MQ_ERR_INVALID_ARG, "%s: unknown rope layout", who);
  if (!std::isfinite(r->factor)) return refuse(MQ_ERR_INVALID_ARG, "%s: rope factor must be finite", who);
  *out = Rope{r->turns, r->rot_dim, r->layout == MQ_ROPE_INTERLEAVED, r->factor};
  return MQ_OK;
}

mq_status check_cache(const char* who, const mq_kv_cache* c, KvCache* out) {
  if (!c) return refuse(MQ_ERR_INVALID_ARG, "%s: null cache", who);
  if (!c->k || !c->v || !c->k_scale || !c->v_scale) return refuse(MQ_ERR_INVALID_ARG, "%s: null pointer in the cache", who);
  if (!on(c->k, 16) || !on(c->v, 16) || !on(c->k_scale, 4) || !on(c->v_scale, 4))
    return refuse(MQ_ERR_INVALID_ARG, "%s: cache codes must be 16-byte and scales 4-byte aligned", who);
  int log2p = 0;
  while (log2p < 8 && (1 << log2p) != c->page_tokens) ++log2p;
  if (log2p < 4 || log2p > 7) return refuse(MQ_ERR_INVALID_ARG, "%s: page_tokens=%d not in {16, 32, 64, 128}", who, c->page_tokens);
  if (c->head_dim < 16 || c->head_dim > 256 || c->head_dim % 16 != 0)
    return refuse(MQ_ERR_INVALID_ARG, "%s: head_dim=%d must be a multiple of 16 in [16, 256]", who, c->head_dim);
  if (c->n_pages < 1 || c->n_pages > 0x7fffffff || c->n_kv_heads < 1)
    return refuse(MQ_ERR_INVALID_ARG, "%s: need 1 <= n_pages < 2^31 and n_kv_heads >= 1", who);
  if (c->n_kv_heads > 1024) return refuse(MQ_ERR_UNSUPPORTED, "%s: more than 1024 key/value heads", who);
  *out = KvCache{c->k, c->v, c->k_scale, c->v_scale, static_cast<int>(c->n_pages), c->page_tokens, log2p, c->n_kv_heads, c->head_dim};
  return MQ_OK;
}

// *empty: a well-formed batch with nothing to do.
mq_status check_batch(const char* who, const mq_kv_batch* b, const KvCache& c, KvBatch* out, bool* empty) {
  if (!b) return refuse(MQ_ERR_INVALID_ARG, "%s: null batch", who);
  if (b->n_seqs < 0 || b->n_rows < 0 || b->max_new < 0 || b->max_len < 0 || b->max_pages < 0)
    return refuse(MQ_ERR_INVALID_ARG, "%s: negative size in the batch", who);
  *empty = b->n_seqs == 0;
  if (*empty) return MQ_OK;
  if (!b->row_start || !b->kv_len || (!b->page_table && b->max_pages > 0)) return refuse(MQ_ERR_INVALID_ARG, "%s: null pointer in the batch", who);
  if (!on(b->row_start, 4) || !on(b->kv_len, 4) || !on(b->page_table, 4))
    return refuse(MQ_ERR_INVALID_ARG, "%s: the batch's arrays must be 4-byte aligned", who);
  if (b->n_seqs > 65535 || b->n_rows > (1 << 28) || b->max_new > (1 << 28) || b->max_pages > (1 << 26) || b->max_len > (1 << 30))
    return refuse(MQ_ERR_UNSUPPORTED, "%s: batch too large", who);
  if (b->max_len > b->max_pages * c.page)
    return refuse(MQ_ERR_INVALID_ARG, "%s: max_len=%lld needs more than max_pages=%lld pages of %d tokens", who,
                  (long long)b->max_len, (long long)b->max_pages, c.page);
  *out = KvBatch{b->row_start, b->kv_len, b->page_table, static_cast<int>(b->n_seqs), static_cast<int>(b->max_pages),
                 static_cast<int>(b->n_rows), static_cast<int>(b->max_new), static_cast<int>(b->max_len)};
  return MQ_OK;
}

// A row of `heads` heads inside a stride, for runs of `run` elements. none: there is no row
// (an empty tensor's address is null).
mq_status check_rows(const char* who, const char* what, const void* p, int64_t stride, int64_t width, int item, int run, bool none) {
  if (!p && !none) return refuse(MQ_ERR_INVALID_ARG, "%s: null %s", who, what);
  if (!on(p, run * item)) return refuse(MQ_ERR_INVALID_ARG, "%s: %s must be %d-byte aligned", who, what, run * item);
  if (stride < width || stride % run != 0)
    return refuse(MQ_ERR_INVALID_ARG, "%s: the row stride of %s must be a multiple of %d, at least %lld", who, what, run,
                  (long long)width);
  if (stride > (int64_t(1) << 31)) return refuse(MQ_ERR_UNSUPPORTED, "%s: the row stride of %s is too large", who, what);
  return MQ_OK;
}

mq_status check_group(const char* who, const KvCache& c, const KvBatch& b, int64_t n_q_heads, int* group) {
  if (n_q_heads < c.heads || n_q_heads % c.heads != 0)
    return refuse(MQ_ERR_INVALID_ARG, "%s: n_q_heads=%lld must be a multiple of n_kv_heads=%d", who, (long long)n_q_heads, c.heads);
  if (n_q_heads > 16384 || int64_t(b.max_new) * (n_q_heads / c.heads) > (1 << 28))
    return refuse(MQ_ERR_UNSUPPORTED, "%s: too many query heads or rows", who);
  *group = static_cast<int>(n_q_heads / c.heads);
  return MQ_OK;
}

}  // namespace

mq_status kv_append_args(const char* who, const mq_kv_cache* cache, const mq_kv_batch* batch, const void* k, const void* v, int dtype,
                         int64_t k_stride, int64_t v_stride, const mq_rope_positions* rope, const int32_t* positions,
                         const void* q, int64_t q_stride, int64_t n_q_heads, void* q_out, AppendArgs* out, bool* nothing) {
  AppendArgs& a = *out;
  a = AppendArgs{};
  bool empty = false;
  mq_status st = check_cache(who, cache, &a.c);
  if (st != MQ_OK) return st;
  if ((st = check_batch(who, batch, a.c, &a.b, &empty)) != MQ_OK) return st;
  if (!is_dtype(dtype)) return refuse(MQ_ERR_INVALID_ARG, "%s: dtype must be MQ_F32 or MQ_BF16", who);
  *nothing = empty || a.b.n_rows == 0 || a.b.max_new == 0;
  const int item = dtype == MQ_F32 ? 4 : 2;
  const int64_t width = int64_t(a.c.heads) * a.c.d;
  if ((st = check_rows(who, "k", k, k_stride, width, item, 4, *nothing)) != MQ_OK) return st;
  if ((st = check_rows(who, "v", v, v_stride, width, item, 4, *nothing)) != MQ_OK) return st;
  if (rope && (st = check_rope(who, rope, a.c.d, 8, &a.rope)) != MQ_OK) return st;
  if (!on(positions, 4)) return refuse(MQ_ERR_INVALID_ARG, "%s: positions must be 4-byte aligned", who);
  if (positions && !rope) return refuse(MQ_ERR_INVALID_ARG, "%s: positions without rope", who);
  if (q) {
    if (n_q_heads < 1 || n_q_heads > 65535) return refuse(MQ_ERR_INVALID_ARG, "%s: n_q_heads must be in [1, 65535]", who);
    if ((st = check_rows(who, "q", q, q_stride, n_q_heads * a.c.d, item, 4, false)) != MQ_OK) return st;
    if (!q_out || !on(q_out, 8)) return refuse(MQ_ERR_INVALID_ARG, "%s: q_out null or not 8-byte aligned", who);
  } else if (q_out) {
    return refuse(MQ_ERR_INVALID_ARG, "%s: q_out without q", who);
  }
  if (*nothing) return MQ_OK;
  a.k = k;
  a.v = v;
  a.q = q;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_stride = q_stride;
  a.positions = positions;
  a.q_out = static_cast<uint16_t*>(q_out);
  a.n_q_heads = static_cast<int>(n_q_heads);
  return MQ_OK;
}

mq_status kv_attention_args(const char* who, const mq_kv_cache* cache, const mq_kv_batch* batch, const void* q, int64_t q_stride,
                            int64_t n_q_heads, float scale, float softcap, int64_t window, void* out, int64_t out_stride, float* lse,
                            void* scratch, size_t scratch_bytes, AttendArgs* out_args, bool* nothing) {
  AttendArgs& a = *out_args;
  a = AttendArgs{};
  bool empty = false;
  mq_status st = check_cache(who, cache, &a.c);
  if (st != MQ_OK) return st;
  if ((st = check_batch(who, batch, a.c, &a.b, &empty)) != MQ_OK) return st;
  if ((st = check_group(who, a.c, a.b, n_q_heads, &a.group)) != MQ_OK) return st;
  if (!std::isfinite(scale)) return refuse(MQ_ERR_INVALID_ARG, "%s: scale must be finite", who);
  if (!(softcap == 0.f || (softcap >= 0x1p-60f && softcap <= 0x1p60f)))
    return refuse(MQ_ERR_INVALID_ARG, "%s: softcap must be 0 (none) or in [2^-60, 2^60]", who);
  if (window < 0) return refuse(MQ_ERR_INVALID_ARG, "%s: window must be >= 0 (0: none)", who);
  *nothing = empty || a.b.n_rows == 0 || a.b.max_new == 0;
  if ((st = check_rows(who, "q", q, q_stride, n_q_heads * a.c.d, 2, 8, *nothing)) != MQ_OK) return st;
  if ((st = check_rows(who, "out", out, out_stride, n_q_heads * a.c.d, 2, 8, *nothing)) != MQ_OK) return st;
  if (!on(lse, 4)) return refuse(MQ_ERR_INVALID_ARG, "%s: lse must be 4-byte aligned", who);
  if (!scratch || !on(scratch, 256)) return refuse(MQ_ERR_INVALID_ARG, "%s: scratch null or not 256-byte aligned", who);
  if (*nothing) return MQ_OK;
  const int sms = sm_count();
  if (scratch_bytes < kv_attention_scratch(a.c, a.b, a.group, sms))
    return refuse(MQ_ERR_INVALID_ARG, "%s: scratch smaller than mq_kv_attention_scratch_bytes", who);
  a.q = static_cast<const uint16_t*>(q);
  a.q_stride = q_stride;
  a.scale = scale;
  a.softcap = softcap;
  a.window = window > (1 << 30) ? 0 : static_cast<int>(window);  // longer than any sequence
  a.out = static_cast<uint16_t*>(out);
  a.out_stride = out_stride;
  a.lse = lse;
  a.scratch = static_cast<uint8_t*>(scratch);
  return MQ_OK;
}

}  // namespace mq

using namespace mq;

extern "C" {

mq_status mq_rope_table(double theta, int rot_dim, int scaling, const double* params, uint64_t* turns, float* factor) try {
  set_last_error("");
  const char* who = "mq_rope_table";
  if (!turns || !factor) return refuse(MQ_ERR_INVALID_ARG, "%s: null output", who);
  if (!(theta > 1.0) || !std::isfinite(theta)) return refuse(MQ_ERR_INVALID_ARG, "%s: theta must be finite and above 1", who);
  if (rot_dim < 2 || rot_dim % 2 != 0 || rot_dim > 4096) return refuse(MQ_ERR_INVALID_ARG, "%s: rot_dim must be even and in [2, 4096]", who);
  if (scaling < MQ_ROPE_PLAIN || scaling > MQ_ROPE_YARN) return refuse(MQ_ERR_INVALID_ARG, "%s: unknown scaling", who);
  const int n_params[4] = {0, 1, 4, 4};
  if (n_params[scaling] && !params) return refuse(MQ_ERR_INVALID_ARG, "%s: this scaling needs params", who);
  for (int i = 0; i < n_params[scaling]; ++i)
    if (!std::isfinite(params[i]) || params[i] <= 0) return refuse(MQ_ERR_INVALID_ARG, "%s: params must be finite and positive", who);
  if (scaling == MQ_ROPE_BANDS && !(params[2] > params[1]))
    return refuse(MQ_ERR_INVALID_ARG, "%s: the high band must lie above the low one", who);
  const long double pi2 = 2 * acosl(-1.0L);
  double low = 0, high = 0;
  *factor = 1.0f;
  if (scaling == MQ_ROPE_YARN) {
    // the pair that makes `b` turns over the original length
    auto pair_of = [&](double b) { return rot_dim * std::log(params[3] / (b * 2 * M_PI)) / (2 * std::log(theta)); };
    low = std::fmax(std::floor(pair_of(params[1])), 0);
    high = std::fmin(std::ceil(pair_of(params[2])), rot_dim - 1);
    if (params[0] > 1) *factor = static_cast<float>(0.1 * std::log(params[0]) + 1.0);
  }
  for (int i = 0; i < rot_dim / 2; ++i) {
    long double w = powl(theta, -2.0L * i / rot_dim);  // radians per position
    if (scaling == MQ_ROPE_LINEAR) {
      w /= params[0];
    } else if (scaling == MQ_ROPE_BANDS) {
      long double keep = (params[3] * w / pi2 - params[1]) / (params[2] - params[1]);
      keep = keep < 0 ? 0 : keep > 1 ? 1 : keep;
      w = w / params[0] * (1 - keep) + w * keep;
    } else if (scaling == MQ_ROPE_YARN) {
      long double keep = 1 - (i - low) / (high > low ? high - low : 0.001);
      keep = keep < 0 ? 0 : keep > 1 ? 1 : keep;
      w = w / params[0] * (1 - keep) + w * keep;
    }
    const long double f = fmodl(w / pi2, 1.0L) * 18446744073709551616.0L;
    turns[i] = f >= 18446744073709551615.0L ? 0 : static_cast<uint64_t>(f + 0.5L);
  }
  return MQ_OK;
} catch (...) {
  return out_of_memory();
}

mq_status mq_rope(const void* x, int x_dtype, int64_t n_rows, int64_t n_heads, int64_t head_dim, int64_t x_stride,
                  const int32_t* positions, const mq_rope_positions* rope, void* y, int y_dtype, int64_t y_stride,
                  void* stream) try {
  TraceRange trace_("mq_rope");
  set_last_error("");
  const char* who = "mq_rope";
  if (!is_dtype(x_dtype) || !is_dtype(y_dtype)) return refuse(MQ_ERR_INVALID_ARG, "%s: dtype must be MQ_F32 or MQ_BF16", who);
  if (n_rows < 0 || n_heads < 1 || head_dim < 2 || head_dim % 2 != 0)
    return refuse(MQ_ERR_INVALID_ARG, "%s: need n_rows >= 0, n_heads >= 1 and an even head_dim >= 2", who);
  if (head_dim > 512 || n_heads > 65535 || n_rows > (int64_t(1) << 31)) return refuse(MQ_ERR_UNSUPPORTED, "%s: sizes too large", who);
  if (!rope) return refuse(MQ_ERR_INVALID_ARG, "%s: null rope", who);
  Rope r{};
  mq_status st = check_rope(who, rope, head_dim, 2, &r);
  if (st != MQ_OK) return st;
  if ((st = check_rows(who, "x", x, x_stride, n_heads * head_dim, x_dtype == MQ_F32 ? 4 : 2, 1, n_rows == 0)) != MQ_OK) return st;
  if ((st = check_rows(who, "y", y, y_stride, n_heads * head_dim, y_dtype == MQ_F32 ? 4 : 2, 1, n_rows == 0)) != MQ_OK) return st;
  if (x && x == y && (x_dtype != y_dtype || x_stride != y_stride))
    return refuse(MQ_ERR_INVALID_ARG, "%s: in place needs one type and one stride", who);
  if ((!positions && n_rows > 0) || !on(positions, 4)) return refuse(MQ_ERR_INVALID_ARG, "%s: positions null or not 4-byte aligned", who);
  if (n_rows == 0) return MQ_OK;
  return finish(launch_rope(x, x_dtype, n_rows, static_cast<int>(n_heads), static_cast<int>(head_dim), x_stride, positions, r, y,
                            y_dtype, y_stride, static_cast<cudaStream_t>(stream), sm_count()), who);
} catch (...) {
  return out_of_memory();
}

mq_status mq_kv_append(const mq_kv_cache* cache, const mq_kv_batch* batch, const void* k, const void* v, int dtype,
                       int64_t k_stride, int64_t v_stride, const mq_rope_positions* rope, const int32_t* positions,
                       const void* q, int64_t q_stride, int64_t n_q_heads, void* q_out, void* stream) try {
  TraceRange trace_("mq_kv_append");
  set_last_error("");
  const char* who = "mq_kv_append";
  AppendArgs a{};
  bool nothing = false;
  const mq_status st = kv_append_args(who, cache, batch, k, v, dtype, k_stride, v_stride, rope, positions, q, q_stride, n_q_heads,
                                      q_out, &a, &nothing);
  if (st != MQ_OK || nothing) return st;
  const cudaError_t e = get_error_word(&a.err);
  if (e != cudaSuccess) return finish(e, who);
  return finish(launch_kv_append(a, dtype, static_cast<cudaStream_t>(stream), sm_count()), who);
} catch (...) {
  return out_of_memory();
}

mq_status mq_kv_read(const mq_kv_cache* cache, const mq_kv_batch* batch, const int32_t* first, const int32_t* out_start,
                     int64_t n_out, int64_t max_out, void* k_out, void* v_out, int dtype, int64_t out_stride, void* stream) try {
  TraceRange trace_("mq_kv_read");
  set_last_error("");
  const char* who = "mq_kv_read";
  ReadArgs a{};
  bool empty = false;
  mq_status st = check_cache(who, cache, &a.c);
  if (st != MQ_OK) return st;
  if ((st = check_batch(who, batch, a.c, &a.b, &empty)) != MQ_OK) return st;
  if (!is_dtype(dtype)) return refuse(MQ_ERR_INVALID_ARG, "%s: dtype must be MQ_F32 or MQ_BF16", who);
  if (n_out < 0 || max_out < 0) return refuse(MQ_ERR_INVALID_ARG, "%s: n_out and max_out must be >= 0", who);
  if (n_out > (1 << 30) || max_out > (1 << 30)) return refuse(MQ_ERR_UNSUPPORTED, "%s: too many rows", who);
  if (empty || n_out == 0 || max_out == 0) return MQ_OK;
  if (!first || !out_start || !on(first, 4) || !on(out_start, 4))
    return refuse(MQ_ERR_INVALID_ARG, "%s: first / out_start null or not 4-byte aligned", who);
  const int item = dtype == MQ_F32 ? 4 : 2;
  const int64_t width = int64_t(a.c.heads) * a.c.d;
  if ((st = check_rows(who, "k_out", k_out, out_stride, width, item, 16 / item, false)) != MQ_OK) return st;
  if ((st = check_rows(who, "v_out", v_out, out_stride, width, item, 16 / item, false)) != MQ_OK) return st;
  a.first = first;
  a.out_start = out_start;
  a.n_out = static_cast<int>(n_out);
  a.max_out = static_cast<int>(max_out);
  a.k_out = k_out;
  a.v_out = v_out;
  a.out_stride = out_stride;
  if (a.b.max_len == 0) return MQ_OK;
  cudaError_t e = get_error_word(&a.err);
  if (e != cudaSuccess) return finish(e, who);
  return finish(launch_kv_read(a, dtype, static_cast<cudaStream_t>(stream)), who);
} catch (...) {
  return out_of_memory();
}

size_t mq_kv_attention_scratch_bytes(const mq_kv_cache* cache, const mq_kv_batch* batch, int64_t n_q_heads) try {
  const char* who = "mq_kv_attention_scratch_bytes";
  set_last_error("");
  KvCache c{};
  KvBatch b{};
  bool empty = false;
  int group = 0;
  if (check_cache(who, cache, &c) != MQ_OK || check_batch(who, batch, c, &b, &empty) != MQ_OK) return 0;
  if (empty) return 256;
  if (check_group(who, c, b, n_q_heads, &group) != MQ_OK) return 0;
  return kv_attention_scratch(c, b, group, sm_count());
} catch (...) {
  out_of_memory();
  return 0;
}

mq_status mq_kv_attention(const mq_kv_cache* cache, const mq_kv_batch* batch, const void* q, int64_t q_stride,
                          int64_t n_q_heads, float scale, float softcap, int64_t window, void* out, int64_t out_stride,
                          float* lse, void* scratch, size_t scratch_bytes, void* stream) try {
  TraceRange trace_("mq_kv_attention");
  set_last_error("");
  const char* who = "mq_kv_attention";
  AttendArgs a{};
  bool nothing = false;
  const mq_status st = kv_attention_args(who, cache, batch, q, q_stride, n_q_heads, scale, softcap, window, out, out_stride, lse,
                                         scratch, scratch_bytes, &a, &nothing);
  if (st != MQ_OK || nothing) return st;
  const cudaError_t e = get_error_word(&a.err);
  if (e != cudaSuccess) return finish(e, who);
  return finish(launch_kv_attention(a, static_cast<cudaStream_t>(stream), sm_count()), who);
} catch (...) {
  return out_of_memory();
}

}  // extern "C"
