// kv_common.cuh — what the key/value cache kernels share: the batch description
// as the device reads it, with every value from device memory checked before it
// is used as an index.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>
#include "internal.h"
#include "ptx.cuh"

namespace qlora {

struct KvBatch {
  const int32_t *token_start;
  const int32_t *kv_len;
  const int32_t *page_table;
  int batch;
  int max_pages;
  int num_pages;
  int page_shift;  // page_size = 1 << page_shift
  int tokens;
  int *dev_err;
};

struct KvSeq {
  int row0;  // first token row of the call
  int n;     // token rows
  int len;   // cached tokens
  __device__ __forceinline__ int pos0() const { return len - n; }  // position of row 0 (negative when len < n)
};

__device__ __forceinline__ void kv_error(const KvBatch &kb) {
  if (kb.dev_err) atomicOr(kb.dev_err, QLORA_DEVERR_KV_INDEX);
}

// Sequence b with its three values clamped to what the buffers hold.
__device__ __forceinline__ KvSeq kv_seq(const KvBatch &kb, int b) {
  const int s0 = kb.token_start[b], s1 = kb.token_start[b + 1], len = kb.kv_len[b];
  const int64_t cap64 = static_cast<int64_t>(kb.max_pages) << kb.page_shift;
  // 2^30 positions at most, so that position - window stays an int
  const int cap = cap64 > (1 << 30) ? 1 << 30 : static_cast<int>(cap64);
  KvSeq q;
  q.row0 = min(max(s0, 0), kb.tokens);
  q.n = min(max(s1, q.row0), kb.tokens) - q.row0;
  q.len = min(max(len, 0), cap);
  if (q.row0 != s0 || q.row0 + q.n != s1 || q.len != len) kv_error(kb);
  return q;
}

// Page of position p (0 <= p < len) of sequence b, or -1 when the table holds no page.
__device__ __forceinline__ int kv_page(const KvBatch &kb, int b, int p) {
  const int pg = __ldg(kb.page_table + static_cast<int64_t>(b) * kb.max_pages + (p >> kb.page_shift));
  return static_cast<unsigned>(pg) < static_cast<unsigned>(kb.num_pages) ? pg : -1;
}

}  // namespace qlora
