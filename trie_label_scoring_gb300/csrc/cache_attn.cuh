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

// mbar_wait for waits that are often not over at once: the limit comes in a
// register instead of a load between two tries. With a negative limit (a test's) the
// kernels begin with barriers that expect an arrival too many, so that the waits for
// pages (streamed) or scores (tiles) never end.
__device__ __forceinline__ long long pipeline_wait_limit() {
  return *const_cast<const volatile long long*>(&g_pipeline_wait_limit);
}
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort_flag, long long limit) {
  const uint32_t a = smem_u32(bar);
  // A try waits a while by itself; most waits that the first does not see out end in
  // the second, which the checks would hold up.
  if (mbar_try_wait(a, parity)) return true;
  const long long t0 = clock64();
  while (true) {
    if (mbar_try_wait(a, parity)) return true;
    if (*abort_flag) return false;
    if (clock64() - t0 > limit) {
      *abort_flag = 1;
      return false;
    }
  }
}

// Four e4m3 codes as two pairs of fp16.
__device__ __forceinline__ void widen4(uint32_t v, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(v));
}
// 16 bytes to shared memory, and this thread's arrival on `bar` once its copies
// have landed (counted in the barrier's expected arrivals).
__device__ __forceinline__ void copy16_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void arrive_after_copies(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ float pow2_byte(uint32_t e) { return __uint_as_float(e << 23); }

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
