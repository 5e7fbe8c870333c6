// Trees of drafted tokens: which nodes are a node's ancestors, and which branch the model
// would have taken.
//
// plan    bits(i) = bits(parent(i)) | bit i; the rotary position is that of the tree's
//         first slot plus the node's depth.
// accept  match(i): draft(i) is the token taken after parent(i), and no earlier child of
//         that parent has it. Node i is right if its whole path matches, bits(i) &
//         ~match = 0: a test of a node's own words, so no walk from the root. The right
//         nodes are one path, node of depth d its d-th. Their rows move to the tree's first
//         slots. Slot d is never the source of a later node (the nodes' indexes ascend along
//         the path and are at least their depths), so a thread that moves its 16 bytes of all
//         rows, loads before stores, in ascending depth, needs no copy in between.
// Both are bound by latency, a few reads that depend on one another: 4 trees of 8 nodes 1.7 us
// (plan) and 3.1 (accept) in a graph; 128 trees of 16 to 64 nodes through 12 layers of 8 heads,
// 3.3 nodes right on the mean, 5.3 us.
#include <algorithm>
#include <atomic>

#include "launch.cuh"
#include "quail_internal.h"
#include "sm103.cuh"
#include "tree.h"

namespace quail {

namespace {

constexpr int kPage = 16;
constexpr int kThreads = 256;

struct Nodes {
  int lo, n, len;
  bool ok;
};
__device__ __forceinline__ Nodes nodes_of(const TreeView& t, int b) {
  Nodes r;
  r.lo = t.offsets[b];
  r.n = t.offsets[b + 1] - r.lo;
  r.len = t.seq_len[b];
  r.ok = r.lo >= 0 && r.n >= 0 && r.n <= t.max_q && r.lo <= t.total - r.n && r.len >= r.n;
  return r;
}

// The nodes are taken 32 at a time, a word of a row. Within such a block a warp doubles the
// paths (a lane's node takes over the bits of the node that its path has come to, five
// times) and finds where each path leaves the block; what lies before is the finished row
// of that node, so the blocks follow one another, all threads copying. A row is built in
// shared memory and written out as whole lines. 256 trees of 300 to 500 nodes (16 words a
// row): 43 us with a thread walking each path and writing its words, 7.8 so.
__global__ void __launch_bounds__(kThreads) tree_plan_kernel(TreeView t, uint32_t* mask, int* rope_pos) {
  extern __shared__ uint32_t s_rows[];  // [nodes, words]
  __shared__ int s_exit[kMaxTree], s_depth[kMaxTree];
  grid_dependency_wait();
  const int b = blockIdx.x, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const Nodes tr = nodes_of(t, b);
  if (!tr.ok) {
    if (threadIdx.x == 0) raise_device_error(t.err, QUAIL_ERR_DEVICE_BOUNDS, b);
    return;
  }
  const int blocks = (tr.n + 31) / 32, words = t.words;
  for (int k = warp; k < blocks; k += kThreads / 32) {
    const int i = 32 * k + lane;
    int p = i < tr.n ? t.parent[tr.lo + i] : -1;
    if (i < tr.n && (p < -1 || p >= i)) {  // no tree: the node stands alone
      raise_device_error(t.err, QUAIL_ERR_DEVICE_BOUNDS, b);
      p = -1;
    }
    uint32_t bits = 1u << lane;
    int at = p >= 32 * k ? p - 32 * k : lane;  // where the path has come to; itself: it leaves the block there
#pragma unroll
    for (int step = 0; step < 5; ++step) {
      bits |= __shfl_sync(0xffffffffu, bits, at);
      at = __shfl_sync(0xffffffffu, at, at);
    }
    const int exit = __shfl_sync(0xffffffffu, p, at);
    if (i < tr.n) {
      s_exit[i] = exit;
      s_depth[i] = __popc(bits);
      s_rows[i * words + k] = bits;
    }
  }
  __syncthreads();
  for (int k = 0; k < blocks; ++k) {
    const int i = 32 * k + threadIdx.x / 8, exit = i < tr.n ? s_exit[i] : -1;  // eight threads a node
    if (i < tr.n)
      for (int w = threadIdx.x % 8; w < k; w += 8)
        s_rows[i * words + w] = w * 32 <= exit ? s_rows[exit * words + w] : 0u;  // a row ends with its node's word
    if (threadIdx.x % 8 == 7 && exit >= 0) s_depth[i] += s_depth[exit];
    __syncthreads();
  }
  uint32_t* out = mask + static_cast<size_t>(tr.lo) * words;
  const int log_w = 32 - __clz(words - 1), w = threadIdx.x & ((1 << log_w) - 1);  // a power of two of threads a row
  if (w < words)
    for (int i = threadIdx.x >> log_w; i < tr.n; i += kThreads >> log_w)
      out[i * words + w] = w <= i / 32 ? s_rows[i * words + w] : 0u;
  for (int i = threadIdx.x; i < tr.n; i += kThreads) rope_pos[tr.lo + i] = tr.len - tr.n + s_depth[i] - 1;
}

constexpr int kAhead = 4;  // rows a thread has on their way

template <bool CODES>
__global__ void __launch_bounds__(kThreads) tree_accept_kernel(AcceptArgs a, const __grid_constant__ LayerPools pools) {
  __shared__ int s_parent[kMaxTree], s_draft[kMaxTree], s_taken[kMaxTree], s_path[kMaxTree];
  __shared__ long long s_src[kMaxTree], s_dst[kMaxTree];  // cache rows of head 0
  __shared__ uint32_t s_match[kMaxTree / 32];
  __shared__ int s_count, s_bad;
  grid_dependency_wait();
  const int b = blockIdx.x;
  const Nodes tr = nodes_of(a.t, b);
  const bool first = blockIdx.y == 0 && a.accepted != nullptr;
  if (!tr.ok) {
    if (threadIdx.x == 0 && first) raise_device_error(a.t.err, QUAIL_ERR_DEVICE_BOUNDS, b);
    return;
  }
  if (threadIdx.x == 0) s_count = s_bad = 0;
  for (int i = threadIdx.x; i < tr.n; i += kThreads) {
    s_parent[i] = a.t.parent[tr.lo + i];
    s_draft[i] = a.draft[tr.lo + i];
    s_taken[i] = a.taken[tr.lo + i];
    s_path[i] = -1;
  }
  __syncthreads();
  for (int i0 = 0; i0 < tr.n; i0 += kThreads) {
    const int i = i0 + threadIdx.x, p = i < tr.n ? s_parent[i] : -1;
    bool match = i == 0;
    if (i > 0 && i < tr.n && p >= 0 && p < i && s_draft[i] == s_taken[p]) {
      match = true;
      for (int j = p + 1; j < i; ++j) match = match && !(s_parent[j] == p && s_draft[j] == s_draft[i]);
    }
    const uint32_t bits = __ballot_sync(0xffffffffu, match);
    if (threadIdx.x % 32 == 0 && i < kMaxTree) s_match[i / 32] = bits;
  }
  __syncthreads();
  const int words = (tr.n + 31) / 32;
  for (int i = threadIdx.x; i < tr.n; i += kThreads) {
    if (!((s_match[i / 32] >> (i % 32)) & 1)) continue;
    const uint32_t* row = a.mask + static_cast<size_t>(tr.lo + i) * a.t.words;
    uint32_t wrong = 0;
    int depth = -1;
    for (int w = 0; w < words; ++w) {
      const uint32_t m = row[w];
      wrong |= m & ~s_match[w];
      depth += __popc(m);
    }
    if (wrong == 0 && depth >= 0 && depth < tr.n) {
      s_path[depth] = i;
      atomicAdd(&s_count, 1);
    }
  }
  __syncthreads();
  const int count = s_count, base = tr.len - tr.n;
  if (first) {
    for (int i = threadIdx.x; i < tr.n; i += kThreads) a.path[tr.lo + i] = s_path[i];
    if (threadIdx.x == 0) {
      a.accepted[b] = count;
      a.new_len[b] = base + count;
      const int last = count > 0 ? s_path[count - 1] : -1;
      a.bonus[b] = last >= 0 ? s_taken[last] : -1;
    }
  }
  if (a.layers == 0) return;
  // ---- the rows' places; d of 1 .. count - 1 (node 0 stays)
  for (int d = threadIdx.x; d < count; d += kThreads) {
    const int from = s_path[d];
    const int* table = a.c.table + static_cast<size_t>(b) * a.c.max_pages;
    auto place = [&](int pos) -> long long {
      const int page = pos / kPage < a.c.max_pages ? table[pos / kPage] : -1;
      if (page < 0 || page >= a.c.num_pages) return -1;
      return (static_cast<long long>(page) * a.c.hkv) * kPage + pos % kPage;
    };
    s_src[d] = from >= 0 ? place(base + from) : -1;
    s_dst[d] = place(base + d);
    if (s_src[d] < 0 || s_dst[d] < 0) s_bad = 1;
  }
  __syncthreads();
  if (s_bad) {
    if (threadIdx.x == 0) raise_device_error(a.t.err, QUAIL_ERR_DEVICE_BOUNDS, b);
    return;
  }
  int d0 = 0;  // the path's first node that moves: up to there slots are right already
  while (d0 < count && s_path[d0] == d0) ++d0;
  if (d0 >= count) return;
  constexpr int kChunks = CODES ? 8 : 16;  // of 16 bytes a row
  const int units = a.layers * 2 * a.c.hkv * kChunks;
  for (int u = blockIdx.y * kThreads + threadIdx.x; u < units; u += gridDim.y * kThreads) {
    const int chunk = u % kChunks, r = u / kChunks, h = r % a.c.hkv, kv = r / a.c.hkv % 2, layer = r / a.c.hkv / 2;
    uint4* pool = reinterpret_cast<uint4*>(pools.p[layer][kv]) + chunk;
    uint8_t* scale = CODES && chunk == 0 ? pools.p[layer][2 + kv] : nullptr;
    const long long head = static_cast<long long>(h) * kPage;
    for (int d = d0; d < count; d += kAhead) {
      uint4 x[kAhead];
      uint8_t e[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (d + k < count) {
          x[k] = pool[(s_src[d + k] + head) * kChunks];
          if (scale != nullptr) e[k] = scale[s_src[d + k] + head];
        }
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (d + k < count) {
          pool[(s_dst[d + k] + head) * kChunks] = x[k];
          if (scale != nullptr) scale[s_dst[d + k] + head] = e[k];
        }
    }
  }
}

}  // namespace

cudaError_t launch_tree_plan(const TreeView& t, uint32_t* mask, int* rope_pos, cudaStream_t st) {
  static std::atomic<bool> configured[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(tree_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxTree * (kMaxTree / 32) * 4);
    if (e != cudaSuccess) return e;
    configured[dev].store(true, std::memory_order_release);
  }
  count_launch();
  const size_t smem = static_cast<size_t>(std::min(t.max_q, t.total)) * t.words * 4;
  return launch_pdl(tree_plan_kernel, dim3(t.num_seqs), dim3(kThreads), smem, st, t, mask, rope_pos);
}

cudaError_t launch_tree_accept(const AcceptArgs& a, const LayerPools& pools, int num_sms, cudaStream_t st) {
  const long long units = 2LL * a.layers * a.c.hkv * (a.c.codes ? 8 : 16);
  const long long shares = (units + kThreads - 1) / kThreads, fill = (8LL * num_sms + a.t.num_seqs - 1) / a.t.num_seqs;
  const dim3 grid(a.t.num_seqs, static_cast<unsigned>(std::max(1LL, std::min(shares, fill))));
  count_launch();
  return a.c.codes ? launch_pdl(tree_accept_kernel<true>, grid, dim3(kThreads), 0, st, a, pools)
                   : launch_pdl(tree_accept_kernel<false>, grid, dim3(kThreads), 0, st, a, pools);
}

}  // namespace quail
