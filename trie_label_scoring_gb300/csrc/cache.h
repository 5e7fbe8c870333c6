// Launch wrappers of the document cache kernels (cache.cu, cache_attention.cu,
// cache_attention_tc.cu). Device pointers throughout; every launch goes to `st` and returns the launch
// status.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "quail_internal.h"

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
  const int* rope_pos = nullptr;  // nullable: the angle goes by pos
  int rotary = 128;               // leading dims of a head that turn
  float magnitude = 1.f;          // of cosine and sine
};
cudaError_t launch_cache_append(const AppendArgs& a, bool f32, int num_sms, cudaStream_t st);
// a.theta, rotary and magnitude follow from d.
cudaError_t launch_cache_append_rope(AppendArgs a, const quail_rope_desc& d, bool f32, int num_sms, cudaStream_t st);

// k_out / v_out [num_tokens, hkv, 128] bf16 (either may be null).
cudaError_t launch_cache_read(const CacheView& c, const int* seq, const int* pos, int num_tokens,
                              __nv_bfloat16* k_out, __nv_bfloat16* v_out, cudaStream_t st);

// The answer token of a letters call, its normed row q | k | v (fp32) the same for
// all n documents: q turned by the documents' lengths (bf16 [n, hq, 128]); and
// attention over the document (o, lse) joined with the token's own key, as rows
// [n, 2 hq 128] of two-term splits.
cudaError_t launch_answer_query(const float* qkv, const int* len, int n, int hq, float theta, __nv_bfloat16* q,
                                cudaStream_t st);
cudaError_t launch_answer_join(const float* qkv, const __nv_bfloat16* o, const float* lse, int n, int hq, int hkv,
                               __nv_bfloat16* out, cudaStream_t st);

// One softmax part of a query row: o = sum 2^(t_j - m_o) v_j and
// l = sum 2^(s_j - m_l), with s the scores in base 2 and t = s, or s plus the
// power of two of key j's value row where v_j are bare codes.
struct __align__(16) PartStat {
  float m_o, m_l, l, pad;
};

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

  // The streaming kernel's work list: prefix_row_tiles x hkv passes over the
  // prefix pages (0: the prefix is not its work), then every sequence's own pages
  // per KV head and row tile, in units of stream_unit_pages, cut into equal chunks
  // over the workers. plan: [0] units, [1] chunk, [2 + b] first unit of sequence b,
  // [2 + num_seqs] past the last.
  bool streamed;
  int prefix_row_tiles;
  long long* plan;
  // Parts, each [rows, 128] fp32 and a PartStat per row; rows are (token, head)
  // except in `cont`, the pieces of work items that began at an earlier worker.
  float* prefix_o;       // pieces that begin a (row tile, head) pass over the prefix
  PartStat* prefix_st;
  float* own_o;          // pieces that begin a sequence's own keys
  PartStat* own_st;
  float* cont_o;         // [workers, kItemRows, 128]
  PartStat* cont_st;

  // The tensor-core tiles' work: the prefix for all rows in prefix_splits key
  // ranges of prefix_split (0: not its work), then every sequence's keys from
  // seq_begin on in seq_splits ranges of seq_split (0: streamed instead).
  // Part s of a row is dense_o[s], the prefix's first; dense_parts 0: a single
  // part, written to out directly, or (clustered) up to eight parts that a cluster of
  // CTAs joins in its shared memory.
  int prefix_split, prefix_splits;
  int seq_begin, seq_split, seq_splits;
  int dense_parts;
  bool clustered;
  float* dense_o;  // [dense_parts, total_q * hq, 128]
  PartStat* dense_st;
};

constexpr int kTileRows = 256;  // query rows of a tensor-core CTA
constexpr int kItemRows = 8;       // query rows of a streaming work item
constexpr int kStreamWarps = 12;   // streaming workers of an SM
// Pages that a streaming worker takes at a time.
__host__ __device__ constexpr int stream_unit_pages(bool codes) { return codes ? 2 : 1; }
cudaError_t launch_attention_stream(const SharedAttnArgs& a, int num_sms, cudaStream_t st);
cudaError_t launch_attention_join(const SharedAttnArgs& a, int num_sms, cudaStream_t st);
cudaError_t launch_attention_prefix(const SharedAttnArgs& a, const CUtensorMap& tmK, const CUtensorMap& tmV,
                                    cudaStream_t st);
cudaError_t launch_attention_sequences(const SharedAttnArgs& a, const CUtensorMap& tmK, const CUtensorMap& tmV,
                                       cudaStream_t st);
cudaError_t set_pipeline_wait_limit_cache_attention(long long cycles);
cudaError_t set_pipeline_wait_limit_cache_attention_tc(long long cycles);

}  // namespace quail
