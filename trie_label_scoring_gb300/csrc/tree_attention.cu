// Attention for trees of drafted tokens over the paged document cache: node i of a
// sequence's n sees the keys [0, len - n) and, of the last n, those that its mask row has
// bits for:  o = softmax(scale q K^T) V,  lse = log sum exp(scale q K^T).
#include "cache_attn.cuh"
#include "launch.cuh"
#include "quail_internal.h"
#include "sm103.cuh"
#include "tree.h"

namespace quail {

namespace {

// One warp per (node, head), four dims a lane, key by key.
__global__ void __launch_bounds__(128) tree_attention_kernel(TreeAttnArgs a) {
  grid_dependency_wait();
  const int b = blockIdx.z, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int h = blockIdx.y * 4 + warp, i = blockIdx.x;
  const int lo = a.q_offsets[b], n = a.q_offsets[b + 1] - lo, len = a.seq_len[b];
  if (lo < 0 || n < 0 || n > a.max_q || lo > a.total_q - n || len < 0 || len > a.max_seq_len || (len > 0 && len < n)) {
    if (threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0) raise_device_error(a.c.err, QUAIL_ERR_DEVICE_BOUNDS, b);
    return;
  }
  if (i >= n || h >= a.hq) return;
  const int g = h / (a.hq / a.c.hkv);
  const size_t row = static_cast<size_t>(lo + i) * a.hq + h;
  const uint2 qu = *reinterpret_cast<const uint2*>(a.q + row * 128 + 4 * lane);
  const float2 q0 = unpack_bf16(qu.x), q1 = unpack_bf16(qu.y);
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k = 0; k < len; ++k) {
    const int j = k - (len - n);
    if (j >= 0 && !((a.mask[static_cast<size_t>(lo + i) * a.words + j / 32] >> (j % 32)) & 1)) continue;
    const int page = a.c.table[static_cast<size_t>(b) * a.c.max_pages + k / kPage];
    if (page < 0 || page >= a.c.num_pages) {
      if (lane == 0) raise_device_error(a.c.err, QUAIL_ERR_DEVICE_BOUNDS, b);
      return;
    }
    const size_t at = (static_cast<size_t>(page) * a.c.hkv + g) * kPage + k % kPage;
    float kx[4], vx[4];
    if (a.c.codes) {
      uint32_t w[2];
      const float ks = pow2_byte(a.c.k_scale[at]), vs = pow2_byte(a.c.v_scale[at]);
      widen4(reinterpret_cast<const uint32_t*>(a.c.k)[at * 32 + lane], w[0], w[1]);
      float2 x = __half22float2(*reinterpret_cast<const __half2*>(&w[0])), y = __half22float2(*reinterpret_cast<const __half2*>(&w[1]));
      kx[0] = x.x * ks; kx[1] = x.y * ks; kx[2] = y.x * ks; kx[3] = y.y * ks;
      widen4(reinterpret_cast<const uint32_t*>(a.c.v)[at * 32 + lane], w[0], w[1]);
      x = __half22float2(*reinterpret_cast<const __half2*>(&w[0])); y = __half22float2(*reinterpret_cast<const __half2*>(&w[1]));
      vx[0] = x.x * vs; vx[1] = x.y * vs; vx[2] = y.x * vs; vx[3] = y.y * vs;
    } else {
      const uint2 ku = reinterpret_cast<const uint2*>(a.c.k)[at * 32 + lane], vu = reinterpret_cast<const uint2*>(a.c.v)[at * 32 + lane];
      float2 x = unpack_bf16(ku.x), y = unpack_bf16(ku.y);
      kx[0] = x.x; kx[1] = x.y; kx[2] = y.x; kx[3] = y.y;
      x = unpack_bf16(vu.x); y = unpack_bf16(vu.y);
      vx[0] = x.x; vx[1] = x.y; vx[2] = y.x; vx[3] = y.y;
    }
    float s = q0.x * kx[0] + q0.y * kx[1] + q1.x * kx[2] + q1.y * kx[3];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    s *= a.scale_log2;
    if (s > m) {
      const float f = exp2f(m - s);
      l *= f;
      o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
      m = s;
    }
    const float p = exp2f(s - m);
    l += p;
    o = make_float4(fmaf(p, vx[0], o.x), fmaf(p, vx[1], o.y), fmaf(p, vx[2], o.z), fmaf(p, vx[3], o.w));
  }
  const bool none = m == -INFINITY && l == 0.f;
  const float f = none ? 0.f : 1.f / l;
  *reinterpret_cast<uint2*>(a.out + row * 128 + 4 * lane) = make_uint2(pack_bf16(o.x * f, o.y * f), pack_bf16(o.z * f, o.w * f));
  if (lane == 0 && a.lse != nullptr) a.lse[row] = none ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

}  // namespace

cudaError_t launch_tree_attention(const TreeAttnArgs& a, int num_sms, cudaStream_t st) {
  count_launch();
  return launch_pdl(tree_attention_kernel, dim3(a.max_q, (a.hq + 3) / 4, a.c.num_seqs), dim3(128), 0, st, a);
}

}  // namespace quail
