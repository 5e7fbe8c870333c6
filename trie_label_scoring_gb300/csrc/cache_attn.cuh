// What the cache attention kernels share: a sequence's queries and keys.
#pragma once
#include "attn_common.cuh"
#include "cache.h"
#include "quail_internal.h"
#include "sm103.cuh"

namespace quail {

constexpr int kPage = 16;

struct QueryRange {
  int lo, hi;  // rows of the sequence's queries
  int len;     // keys
  bool ok;
};

__device__ __forceinline__ QueryRange query_range(const SharedAttnArgs& a, int b) {
  QueryRange r;
  r.lo = a.q_offsets ? a.q_offsets[b] : b;
  r.hi = a.q_offsets ? a.q_offsets[b + 1] : b + 1;
  r.len = a.seq_len[b];
  const int n = r.hi - r.lo;
  r.ok = r.lo >= 0 && n >= 0 && n <= a.max_q && r.hi <= a.total_q && r.len >= 0 && r.len <= a.max_seq_len &&
         (r.len == 0 || r.len - (a.causal ? n : 0) >= a.prefix_len);
  return r;
}

// Pages of sequence b's own keys that its queries read (0: none, or a bad sequence).
__device__ __forceinline__ int own_pages(const SharedAttnArgs& a, int b) {
  const QueryRange r = query_range(a, b);
  return r.ok && r.hi > r.lo && r.len > a.prefix_len ? (r.len - a.prefix_len + kPage - 1) / kPage : 0;
}

// Keys that row r (counted within the sequence's rows of one KV head) sees.
__device__ __forceinline__ int row_limit(const SharedAttnArgs& a, const QueryRange& q, int r) {
  return a.causal ? q.len - (q.hi - q.lo) + r / (a.hq / a.c.hkv) + 1 : q.len;
}

// Past the last key that any row of the tensor-core tile holding row r sees.
__device__ __forceinline__ int tile_key_end(const SharedAttnArgs& a, const QueryRange& q, int r) {
  const int n = (q.hi - q.lo) * (a.hq / a.c.hkv);
  return row_limit(a, q, min(n, (r / kTileRows + 1) * kTileRows) - 1);
}

}  // namespace quail
