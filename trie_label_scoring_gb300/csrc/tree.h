// Launch wrappers of the kernels for trees of drafted tokens over the document cache:
// page tables that follow the lengths (cache_pages.cu), masks and verdicts (tree.cu),
// attention (tree_attention.cu). Device pointers throughout; every launch goes to `st`
// and returns the launch status.
#pragma once
#include "cache.h"

namespace quail {

constexpr int kMaxTree = 1024;  // nodes of a tree

struct ResizeArgs {
  CacheView c;
  int* table;               // c.table, written
  const int* prefix_pages;  // [prefix_len / 16]
  int prefix_len;           // a multiple of 16
  const int* old_len;
  const int* new_len;
  int* ring;   // [num_pages]
  int* state;  // head, count, a counter that is 0 between calls, unused
  int* granted;
  int* offsets;  // [num_seqs + 1]
  int* token_seq;  // nullable, with token_pos
  int* token_pos;
  int max_tokens;
};
cudaError_t launch_cache_resize(const ResizeArgs& a, int num_sms, cudaStream_t st);

// The trees of a batch: sequence b's nodes are rows [offsets[b], offsets[b + 1]).
struct TreeView {
  const int* parent;  // [total], within the tree, -1: none
  const int* offsets;
  const int* seq_len;
  int num_seqs, total, max_q;
  int words;  // of a mask row, (max_q + 31) / 32
  int* err;
};
cudaError_t launch_tree_plan(const TreeView& t, uint32_t* mask, int* rope_pos, cudaStream_t st);

constexpr int kAcceptLayers = 128;  // of one launch
struct LayerPools {
  uint8_t* p[kAcceptLayers][4];  // k, v, k_scale, v_scale
};
struct AcceptArgs {
  TreeView t;
  CacheView c;  // pointers of the layers apart
  int layers;
  const uint32_t* mask;
  const int* draft;
  const int* taken;
  int* path;
  // nullptr, with what follows and path: a later launch of the same call, which moves rows only
  int* accepted;
  int* new_len;
  int* bonus;
};
cudaError_t launch_tree_accept(const AcceptArgs& a, const LayerPools& pools, int num_sms, cudaStream_t st);

struct SharedItem {
  int row0, tokens;  // first node's row, nodes
  int g;             // KV head
  int parts;         // CTAs that have one, this and those after it; 0: no item
};

struct TreeAttnArgs {
  CacheView c;
  int hq;
  const __nv_bfloat16* q;  // [total_q, hq, 128]
  const int* q_offsets;
  int total_q, max_q;
  const int* seq_len;
  int max_seq_len;
  const uint32_t* mask;  // [total_q, words]
  int words;
  float scale_log2;  // score factor times log2(e)
  __nv_bfloat16* out;
  float* lse;  // nullable

  int tile_cols;    // query columns of a tile: 16, 32, 64, 96 or 128
  int tile_tokens;  // nodes of a tile, tile_cols / (hq / hkv)
  int ctas;
  bool direct;  // whole (sequence, head, tile) items by turns; else equal runs of the work list
  // of the runs: the item that each CTA begins and leaves; two parts of a CTA, of tile_cols
  // rows of 128 each: what it did of that item, and what it did of one begun before it
  SharedItem* shared_items;
  float* part_o;
  PartStat* part_st;
};
cudaError_t launch_tree_attention(const TreeAttnArgs& a, const CUtensorMap& tmK, const CUtensorMap& tmV,
                                  const CUtensorMap& tmQ, cudaStream_t st);
cudaError_t set_pipeline_wait_limit_tree_attention(long long cycles);

}  // namespace quail
