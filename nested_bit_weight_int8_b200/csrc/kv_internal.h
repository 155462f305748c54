// The paged 8-bit key/value cache and the rotary positions as the kernels see
// them (kv_cache.cu, kv_attention.cu), and the launchers behind the entry
// points of kv_api.cu.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>
#include <vector>

#include "../../include/mq.h"

namespace mq {

// One layer's cache: pages of `page` tokens, each page and key/value head one
// contiguous tile of page x d bytes (byte = code + 128) with one fp32 scale.
struct KvCache {
  uint8_t* k;
  uint8_t* v;
  float* k_scale;  // n_pages x heads
  float* v_scale;
  int n_pages;
  int page;      // tokens per page: 16, 32, 64 or 128
  int page_log2;
  int heads;
  int d;
};

// The rows of one call, by sequence (device arrays).
struct KvBatch {
  const int32_t* row_start;  // n_seqs + 1
  const int32_t* kv_len;     // n_seqs, the new rows included
  const int32_t* pages;      // n_seqs x max_pages
  int n_seqs;
  int max_pages;
  int n_rows;
  int max_new;
  int max_len;
};

// Rotary positions: angle of pair i at position p = 2 pi frac(p turns[i] / 2^64).
struct Rope {
  const uint64_t* turns;  // rot / 2; null: no rotation
  int rot;
  int interleaved;
  float factor;
};

struct AppendArgs {
  KvCache c;
  KvBatch b;
  Rope rope;
  const void* k;
  const void* v;
  const void* q;       // null: no queries
  int64_t k_stride, v_stride, q_stride;  // elements between rows
  const int32_t* positions;              // null: a token's place in its sequence
  uint16_t* q_out;     // n_rows x n_q_heads x d bf16
  int n_q_heads;
  uint32_t* err;
};

struct ReadArgs {
  KvCache c;
  KvBatch b;
  const int32_t* first;      // n_seqs
  const int32_t* out_start;  // n_seqs + 1
  int n_out, max_out;
  void* k_out;
  void* v_out;
  int64_t out_stride;
  uint32_t* err;
};

struct AttendArgs {
  KvCache c;
  KvBatch b;
  const uint16_t* q;  // bf16
  int64_t q_stride;
  int group;          // query heads per key/value head
  float scale;
  float softcap;      // 0: none
  int window;         // 0: none
  uint16_t* out;      // bf16
  int64_t out_stride;
  float* lse;         // n_rows x (heads * group), or null
  uint8_t* scratch;
  uint32_t* err;
};

cudaError_t launch_rope(const void* x, int x_dtype, int64_t rows, int heads, int d, int64_t x_stride,
                        const int32_t* positions, const Rope& rope, void* y, int y_dtype, int64_t y_stride,
                        cudaStream_t stream, int sms);
cudaError_t launch_kv_append(const AppendArgs& a, int dtype, cudaStream_t stream, int sms);
cudaError_t launch_kv_read(const ReadArgs& a, int dtype, cudaStream_t stream);
size_t kv_attention_scratch(const KvCache& c, const KvBatch& b, int group, int sms);
// Sequences with more than `limit` rows (query tokens times heads of a group).
// Launched directly behind kv_attend_kernel, whose shared rows (`few`) it joins with its own.
// `scratch`: kv_prompt_scratch bytes.
struct Scratch;
size_t kv_prompt_scratch(const KvCache& c, const KvBatch& b, int group, int sms);
cudaError_t launch_kv_prompt(const AttendArgs& a, int limit, const Scratch& few, uint8_t* scratch, cudaStream_t stream, int sms);
cudaError_t launch_kv_attention(const AttendArgs& a, cudaStream_t stream, int sms);

// A chained stack's attention: each layer's launch arguments.
struct ChainCached {
  std::vector<AppendArgs> append;
  std::vector<AttendArgs> attend;
};

// The checks of mq_kv_append and mq_kv_attention, and their launch arguments but
// for the error word. *nothing: a well-formed call that has nothing to do.
mq_status kv_append_args(const char* who, const mq_kv_cache* cache, const mq_kv_batch* batch, const void* k, const void* v, int dtype,
                         int64_t k_stride, int64_t v_stride, const mq_rope_positions* rope, const int32_t* positions,
                         const void* q, int64_t q_stride, int64_t n_q_heads, void* q_out, AppendArgs* out, bool* nothing);
mq_status kv_attention_args(const char* who, const mq_kv_cache* cache, const mq_kv_batch* batch, const void* q, int64_t q_stride,
                            int64_t n_q_heads, float scale, float softcap, int64_t window, void* out, int64_t out_stride, float* lse,
                            void* scratch, size_t scratch_bytes, AttendArgs* out_args, bool* nothing);

#ifdef __CUDACC__
// These kernels may be resident while the one before them still writes what they read: they
// wait for it (pdl_wait_primary), and read with plain loads. The read-only path (__ldg, const
// __restrict__) is for memory that nothing writes while a kernel lives.
//
// A sequence of the batch: its first row, its rows and its tokens. A sequence
// whose numbers do not fit the call (rows outside [0, n_rows), more rows than
// max_new, more tokens than max_len) is flagged and has no rows.
struct Seq {
  int r0, n, len;
};
__device__ __forceinline__ Seq load_seq(const KvBatch& b, int s, uint32_t* err) {
  Seq q;
  q.r0 = b.row_start[s];
  q.n = b.row_start[s + 1] - q.r0;
  q.len = b.kv_len[s];
  if (q.r0 < 0 || q.n < 0 || q.n > b.max_new || q.r0 > b.n_rows - q.n || q.len > b.max_len) {
    if (err) atomicOr(err, 16u);  // kErrBounds
    q.n = 0;
    q.len = 0;
  }
  q.len = q.len < 0 ? 0 : q.len;
  return q;
}
// The page that holds token `index * page` of sequence s, or -1 (flagged)
// where the table names none.
__device__ __forceinline__ int load_page(const KvCache& c, const KvBatch& b, int s, int index, uint32_t* err) {
  const int p = b.pages[int64_t(s) * b.max_pages + index];
  if (p >= 0 && p < c.n_pages) return p;
  atomicOr(err, 16u);
  return -1;
}
#endif

}  // namespace mq
