// Launch wrappers of the document cache kernels (cache.cu, cache_attention.cu,
// cache_attention_tc.cu). Device pointers throughout; every launch goes to
// `st` and returns the launch status.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace quail {

// A paged K/V pool and its page table. codes: one byte an element plus one
// biased exponent byte per (page, head, slot); else bf16 elements.
struct CacheView {
  void* k;
  void* v;
  uint8_t* k_scale;
  uint8_t* v_scale;
  bool codes;
  int hkv;
  int num_pages;
  int num_seqs, max_pages;
  const int* table;  // [num_seqs, max_pages]
  int* err;
};

struct AppendArgs {
  CacheView c;
  const void* qkv;  // [num_tokens, (hq + 2 hkv) * 128], row stride ld
  long long ld;
  int num_tokens, hq;
  const int* seq;
  const int* pos;
  const __nv_bfloat16* gq;  // nullable: no norm
  const __nv_bfloat16* gk;
  float eps;
  float theta;  // 0: no rotation
  __nv_bfloat16* q_out;  // nullable
};
cudaError_t launch_cache_append(const AppendArgs& a, bool f32, cudaStream_t st);

// k_out / v_out [num_tokens, hkv, 128] bf16 (either may be null).
cudaError_t launch_cache_read(const CacheView& c, const int* seq, const int* pos, int num_tokens,
                              __nv_bfloat16* k_out, __nv_bfloat16* v_out, cudaStream_t st);

struct SharedAttnArgs {
  CacheView c;
  int hq;
  const __nv_bfloat16* q;  // [total_q, hq, 128]
  const int* q_offsets;    // nullable: sequence b's only query is row b
  int total_q, max_q;
  const int* seq_len;
  int max_seq_len;
  const int* prefix_pages;
  int prefix_len;  // a multiple of 16
  int causal;
  float scale_log2;  // score factor times log2(e)
  __nv_bfloat16* out;
  float* lse;  // nullable
};
cudaError_t launch_attention_simple(const SharedAttnArgs& a, cudaStream_t st);

}  // namespace quail
