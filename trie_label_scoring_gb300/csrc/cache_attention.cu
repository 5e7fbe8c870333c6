// Attention over the paged document cache for a batch whose sequences share
// their first prefix_len tokens:
//   o = softmax(scale q K^T) V,  lse = log sum exp(scale q K^T)
#include <cuda_fp8.h>

#include "attn_common.cuh"
#include "cache.h"
#include "launch.cuh"
#include "quail_internal.h"
#include "sm103.cuh"

namespace quail {

namespace {

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

// Block = (query of a sequence, KV head), one warp per query head of the group.
__global__ void attention_simple_kernel(SharedAttnArgs a) {
  grid_dependency_wait();
  const int b = blockIdx.z, g = blockIdx.y, i = blockIdx.x;
  const QueryRange r = query_range(a, b);
  const int G = a.hq / a.c.hkv, lane = threadIdx.x & 31;
  if (!r.ok) {
    if (threadIdx.x == 0) raise_device_error(a.c.err, QUAIL_ERR_DEVICE_BOUNDS, b);
    return;
  }
  if (i >= r.hi - r.lo) return;
  const size_t row = r.lo + i;
  const int n = a.causal && r.len > 0 ? r.len - (r.hi - r.lo) + i + 1 : r.len;
  for (int hl = threadIdx.x >> 5; hl < G; hl += blockDim.x >> 5) {
    const size_t h = row * a.hq + g * G + hl;
    float q[4];
    for (int d = 0; d < 4; ++d) q[d] = __bfloat162float(a.q[h * 128 + 4 * lane + d]);
    float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int j = 0; j < n; ++j) {
      const int page = j < a.prefix_len ? a.prefix_pages[j / kPage]
                                        : a.c.table[static_cast<size_t>(b) * a.c.max_pages + j / kPage];
      if (page < 0 || page >= a.c.num_pages) {
        raise_device_error(a.c.err, QUAIL_ERR_DEVICE_BOUNDS, b);
        return;
      }
      const size_t at = (static_cast<size_t>(page) * a.c.hkv + g) * kPage + j % kPage;
      float k[4], v[4];
      for (int d = 0; d < 4; ++d) {
        const size_t e = at * 128 + 4 * lane + d;
        if (a.c.codes) {
          __nv_fp8_e4m3 kc, vc;
          kc.__x = static_cast<const uint8_t*>(a.c.k)[e];
          vc.__x = static_cast<const uint8_t*>(a.c.v)[e];
          k[d] = static_cast<float>(kc) * __uint_as_float(static_cast<uint32_t>(a.c.k_scale[at]) << 23);
          v[d] = static_cast<float>(vc) * __uint_as_float(static_cast<uint32_t>(a.c.v_scale[at]) << 23);
        } else {
          k[d] = __bfloat162float(static_cast<const bf16*>(a.c.k)[e]);
          v[d] = __bfloat162float(static_cast<const bf16*>(a.c.v)[e]);
        }
      }
      float s = q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3];
      for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
      s *= a.scale_log2;
      const float nm = fmaxf(m, s);
      const float ref = nm == -INFINITY ? 0.f : nm;
      const float f = exp2f(m - ref), p = exp2f(s - ref);
      m = nm;
      l = l * f + p;
      for (int d = 0; d < 4; ++d) o[d] = o[d] * f + p * v[d];
    }
    for (int d = 0; d < 4; ++d) a.out[h * 128 + 4 * lane + d] = __float2bfloat16(n > 0 ? o[d] / l : 0.f);
    if (lane == 0 && a.lse) a.lse[h] = n > 0 ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
  }
}

}  // namespace

cudaError_t launch_attention_simple(const SharedAttnArgs& a, cudaStream_t st) {
  if (a.total_q <= 0 || a.c.num_seqs <= 0) return cudaSuccess;
  count_launch();
  return launch_pdl(attention_simple_kernel, dim3(a.max_q, a.c.hkv, a.c.num_seqs), dim3(128), 0, st, a);
}

}  // namespace quail
