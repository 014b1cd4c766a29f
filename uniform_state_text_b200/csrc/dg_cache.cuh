// Device view of a paged key/value cache and of a batch of new tokens, shared
// by the cache and attention kernels. Every index that comes from device
// memory (page numbers, lengths, token offsets) is checked here before it
// forms an address.
#pragma once
#include <stdint.h>

#include "dg.h"
#include "dg_common.cuh"

namespace dg {

constexpr int kMaxBatch = 1024;

// Grid-constant copy of dg_kv_cache and dg_kv_batch.
struct KvView {
  dg_kv_cache c;
  dg_kv_batch b;
};

// DG_EINVAL or DG_ETIMEOUT into the cache's status word (the first one stays).
__device__ __forceinline__ void raise_status(int* status, int code) { atomicCAS(status, 0, code); }

// Row (page, head, offset) of position `pos` of a sequence whose page table
// entries are `table`; -1 if the position has no page (the status is raised).
// The host has checked that the cache has fewer than 2^31 rows.
__device__ __forceinline__ int kv_row(const KvView& w, const int32_t* table, int64_t pos, int head) {
  if (pos >= 0 && pos <= 0x7fffffff) {         // the table covers fewer than 2^31 positions
    const uint32_t at = (uint32_t)pos / (uint32_t)w.c.page_size;
    if (at < (uint32_t)w.b.table_stride) {
      const int page = __ldg(table + at);
      if (page >= 0 && page < w.c.pages)
        return (page * w.c.kv_heads + head) * w.c.page_size + (int)((uint32_t)pos - at * (uint32_t)w.c.page_size);
    }
  }
  raise_status(w.c.status, DG_EINVAL);
  return -1;
}

// Sequence of a token: the last b with first[b] <= token; -1 for padding rows.
__device__ __forceinline__ int kv_sequence(const KvView& w, int token) {
  int lo = 0, hi = w.b.batch;            // first[lo] <= token < first[hi] is sought
  if (token < __ldg(w.b.first) || token >= __ldg(w.b.first + hi)) return -1;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(w.b.first + mid) <= token) lo = mid;
    else hi = mid;
  }
  return lo;
}

// New tokens [*t0, *t0 + n) of sequence b (n returned), held to the rows that exist.
__device__ __forceinline__ int kv_new(const KvView& w, int b, int* t0) {
  const int lo = max(0, min(__ldg(w.b.first + b), w.b.tokens));
  const int hi = max(lo, min(__ldg(w.b.first + b + 1), w.b.tokens));
  *t0 = lo;
  return hi - lo;
}

// Cached positions before sequence b's new tokens, held to what its page table
// can name: a length beyond it (or below zero) is an error, not a long loop.
__device__ __forceinline__ int kv_past(const KvView& w, int b, int n) {
  const int past = __ldg(w.b.past + b);
  const int room = max(0, w.b.table_stride * w.c.page_size - n);   // the product is below 2^31
  if (past < 0 || past > room) raise_status(w.c.status, DG_EINVAL);
  return max(0, min(past, room));
}

}  // namespace dg
