// Writing and reading the paged document cache.
//
// Append, per token and head row x of 128 (q and k heads; v passes through):
//   y = x / sqrt(mean(x^2) + eps) * g,  then pair (j, j + 64) turned by
//   pos * theta^(-2j/128); k and v go to slot pos % 16 of the token's page.
// An 8-bit cache holds e4m3 codes c and one power of two 2^e per (token, head),
// the smallest with max |x| <= 448 * 2^e: x ~ c * 2^e. A power of two costs no
// precision (e4m3 keeps 4 significant bits wherever the value falls, short of
// its subnormals) and makes every c * 2^e a bf16 value exactly, so reading the
// cache back, or attending to it, rounds nothing.
//
// Both kernels are bound by HBM: no element is touched twice. Eight lanes take
// one head row, lane i the elements 8i..8i+7 and 64+8i..64+8i+7, so both
// members of a rotated pair sit in one thread, every load and store is a
// 16-byte piece of a full 128-byte line, and the row sums take three shuffles.
#include <cuda_fp8.h>

#include "attn_common.cuh"
#include "cache.h"
#include "launch.cuh"
#include "quail_internal.h"
#include "sm103.cuh"

namespace quail {

namespace {

constexpr int kPage = 16;
constexpr int kRowLanes = 8;

__device__ __forceinline__ uint4 ldg_stream(const void* p) { return __ldcs(reinterpret_cast<const uint4*>(p)); }

__device__ __forceinline__ void widen8(const uint4& u, float* x) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack_bf16(w[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

// x[0..7] = dims 8l.., x[8..15] = dims 64 + 8l.. of the head row at p.
template <typename T>
__device__ __forceinline__ void load_row(const T* p, int l, float (&x)[16]);
template <>
__device__ __forceinline__ void load_row<bf16>(const bf16* p, int l, float (&x)[16]) {
  const uint4 a = ldg_stream(p + 8 * l), b = ldg_stream(p + 64 + 8 * l);
  widen8(a, x);
  widen8(b, x + 8);
}
template <>
__device__ __forceinline__ void load_row<float>(const float* p, int l, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 f = __ldcs(reinterpret_cast<const float4*>(p + (i < 2 ? 0 : 64) + 8 * l + 4 * (i & 1)));
    x[4 * i] = f.x;
    x[4 * i + 1] = f.y;
    x[4 * i + 2] = f.z;
    x[4 * i + 3] = f.w;
  }
}

__device__ __forceinline__ void store_row_bf16(bf16* p, int l, const float (&x)[16]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float* y = x + 8 * h;
    *reinterpret_cast<uint4*>(p + 64 * h + 8 * l) =
        make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
  }
}

// Sum / maximum over the eight lanes of a row.
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = 1; o < kRowLanes; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float row_max(float v) {
#pragma unroll
  for (int o = 1; o < kRowLanes; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Biased exponent of the smallest 2^e with amax <= 448 * 2^e = 1.75 * 2^(e+8),
// from amax's own exponent and whether its fraction is above 0.75; at least
// 2^-100, so that every code times 2^e is a normal or subnormal bf16.
constexpr int kMinScale = 27;
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = static_cast<int>(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e < kMinScale ? kMinScale : e;
}

// Row x as codes and scale; m is the row's largest finite |x|. An infinity
// saturates to +-448 * 2^e, a NaN stays one.
__device__ __forceinline__ void store_row_codes(uint8_t* p, uint8_t* scale, int l, const float (&x)[16], float m) {
  const int e = scale_exponent(m);
  const float inv = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float* y = x + 8 * h + 4 * i;
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(y[0] * inv, y[1] * inv), __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(y[2] * inv, y[3] * inv), __NV_SATFINITE, __NV_E4M3);
      w[i] = lo | hi << 16;
    }
    *reinterpret_cast<uint2*>(p + 64 * h + 8 * l) = make_uint2(w[0], w[1]);
  }
  if (l == 0) *scale = static_cast<uint8_t>(e);
}

// Physical page of position pos of sequence seq, or -1 (error recorded).
__device__ __forceinline__ int page_of(const CacheView& c, int seq, int pos, int token) {
  int page = -1;
  if (seq < c.num_seqs && pos >= 0 && pos / kPage < c.max_pages)
    page = c.table[static_cast<size_t>(seq) * c.max_pages + pos / kPage];
  if (page < 0 || page >= c.num_pages) {
    raise_device_error(c.err, QUAIL_ERR_DEVICE_BOUNDS, token);
    return -1;
  }
  return page;
}

// ------------------------------------------------------------------ append
// Block = one token: 16 row groups of eight lanes walk its hq + 2 hkv heads,
// so the 64 angles of a position are computed once per group and shared by
// the heads that the group takes.
constexpr int kAppendThreads = 128;
constexpr int kAppendGroups = kAppendThreads / kRowLanes;

template <typename T>
__global__ void __launch_bounds__(kAppendThreads) cache_append_kernel(AppendArgs a, RopeTable rt) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int t = blockIdx.x;
  const int group = threadIdx.x / kRowLanes, l = threadIdx.x % kRowLanes;
  const int seq = a.seq[t];
  if (seq < 0) return;  // a padding token: nothing of it is written
  const int pos = a.pos[t];
  const int page = page_of(a.c, seq, pos, t);
  if (page < 0) return;
  const int heads = a.hq + 2 * a.c.hkv;
  const T* row = static_cast<const T*>(a.qkv) + static_cast<long long>(t) * a.ld;
  float cs[8], sn[8];
  if (a.theta > 0.f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) rope_cs(pos, rt.w[8 * l + i], cs[i], sn[i]);
  }
  // whole warps take the loop together: the row sums shuffle over all lanes
  for (int h0 = 0; h0 < heads; h0 += kAppendGroups) {
    const int h = h0 + group;
    const bool live = h < heads;
    const bool is_q = h < a.hq, is_k = !is_q && h < a.hq + a.c.hkv;
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = 0.f;
    if (live) load_row(row + h * 128, l, x);
    const bf16* gain = is_q ? a.gq : is_k ? a.gk : nullptr;
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) ss = fmaf(x[i], x[i], ss);
    ss = row_sum(ss);
    if (gain != nullptr) {
      const float r = rsqrtf(ss * (1.f / 128.f) + a.eps);
      float g[16];
      widen8(*reinterpret_cast<const uint4*>(gain + 8 * l), g);
      widen8(*reinterpret_cast<const uint4*>(gain + 64 + 8 * l), g + 8);
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = x[i] * r * g[i];
    }
    if (a.theta > 0.f && (is_q || is_k)) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float x1 = x[i], x2 = x[i + 8];
        x[i] = x1 * cs[i] - x2 * sn[i];
        x[i + 8] = x2 * cs[i] + x1 * sn[i];
      }
    }
    if (live && is_q) {
      if (a.q_out != nullptr) store_row_bf16(a.q_out + (static_cast<size_t>(t) * a.hq + h) * 128, l, x);
    }
    // the codes' row maximum shuffles: every lane of the warp goes through it
    const int g = h - a.hq - (is_k ? 0 : a.c.hkv);
    const size_t at = (static_cast<size_t>(page) * a.c.hkv + g) * kPage + pos % kPage;
    const bool kv = live && !is_q;
    if (!a.c.codes) {
      if (kv) store_row_bf16(static_cast<bf16*>(is_k ? a.c.k : a.c.v) + at * 128, l, x);
    } else {
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float v = fabsf(x[i]);
        m = fmaxf(m, v < INFINITY ? v : 0.f);
      }
      m = row_max(m);
      if (kv) store_row_codes(static_cast<uint8_t*>(is_k ? a.c.k : a.c.v) + at * 128,
                              (is_k ? a.c.k_scale : a.c.v_scale) + at, l, x, m);
    }
  }
}

// ------------------------------------------------------------------ read
// Eight lanes per (token, K or V, head) row.
constexpr int kReadThreads = 256;
constexpr int kReadGroups = kReadThreads / kRowLanes;

__device__ __forceinline__ uint32_t codes_to_bf16x2(uint32_t two, float scale) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two & 0xffffu), __NV_E4M3);
  const float2 f = __half22float2(__half2(h));
  return pack_bf16(f.x * scale, f.y * scale);
}

// Elements 16 l .. 16 l + 15 of a row: sixteen codes w times sc.
__device__ __forceinline__ void store_codes_bf16(bf16* out, int l, const uint4& w, float sc) {
  const uint32_t in[4] = {w.x, w.y, w.z, w.w};
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[2 * i] = codes_to_bf16x2(in[i], sc);
    o[2 * i + 1] = codes_to_bf16x2(in[i] >> 16, sc);
  }
  *reinterpret_cast<uint4*>(out + 16 * l) = make_uint4(o[0], o[1], o[2], o[3]);
  *reinterpret_cast<uint4*>(out + 16 * l + 8) = make_uint4(o[4], o[5], o[6], o[7]);
}

__global__ void __launch_bounds__(kReadThreads)
    cache_read_kernel(CacheView c, const int* seq, const int* pos, int num_tokens, bf16* k_out, bf16* v_out) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int l = threadIdx.x % kRowLanes;
  const long long u = static_cast<long long>(blockIdx.x) * kReadGroups + threadIdx.x / kRowLanes;
  const int per = 2 * c.hkv;
  const int t = static_cast<int>(u / per), r = static_cast<int>(u % per);
  if (t >= num_tokens) return;
  const int s = seq[t];
  if (s < 0) return;
  const int p = pos[t];
  const int page = page_of(c, s, p, t);
  if (page < 0) return;
  const bool is_k = r < c.hkv;
  const int h = is_k ? r : r - c.hkv;
  bf16* out = is_k ? k_out : v_out;
  if (out == nullptr) return;
  out += (static_cast<size_t>(t) * c.hkv + h) * 128;
  const size_t at = (static_cast<size_t>(page) * c.hkv + h) * kPage + p % kPage;
  if (!c.codes) {
    const bf16* in = static_cast<const bf16*>(is_k ? c.k : c.v) + at * 128;
    const uint4 a = ldg_stream(in + 8 * l), b = ldg_stream(in + 64 + 8 * l);
    *reinterpret_cast<uint4*>(out + 8 * l) = a;
    *reinterpret_cast<uint4*>(out + 64 + 8 * l) = b;
  } else {
    const uint4 w = ldg_stream(static_cast<const uint8_t*>(is_k ? c.k : c.v) + at * 128 + 16 * l);
    const int e = (is_k ? c.k_scale : c.v_scale)[at];
    const float sc = __uint_as_float(static_cast<uint32_t>(e) << 23);
    store_codes_bf16(out, l, w, sc);
  }
}

// ------------------------------------------------------------------ widen
// Block = one page of the list (the prefix, then wide_own pages per sequence):
// its K and V rows as bf16 for the tensor-core tiles. Exact, and small next to
// their work: the tiles have 256 rows to multiply with every key.
__global__ void __launch_bounds__(kReadThreads) cache_widen_kernel(SharedAttnArgs a) {
  grid_dependency_wait();
  const int pp = a.prefix_len / kPage, p = blockIdx.x;
  int page;
  if (p < pp) {
    page = a.prefix_pages[p];
  } else {
    const int b = (p - pp) / a.wide_own, j = (p - pp) % a.wide_own;
    const int len = a.seq_len[b];
    if (len > a.max_seq_len || (pp + j) * kPage >= len) return;
    page = a.c.table[static_cast<size_t>(b) * a.c.max_pages + pp + j];
  }
  if (page < 0 || page >= a.c.num_pages) {
    if (threadIdx.x == 0) raise_device_error(a.c.err, QUAIL_ERR_DEVICE_BOUNDS, p);
    return;  // the rows that read this page are void
  }
  const int l = threadIdx.x % kRowLanes;
  const int rows = a.c.hkv * kPage;
  for (int u = threadIdx.x / kRowLanes; u < 2 * rows; u += kReadGroups) {
    const bool is_k = u < rows;
    const int r = is_k ? u : u - rows;
    const size_t at = static_cast<size_t>(page) * rows + r;
    const uint4 w = ldg_stream(static_cast<const uint8_t*>(is_k ? a.c.k : a.c.v) + at * 128 + 16 * l);
    const float sc = __uint_as_float(static_cast<uint32_t>((is_k ? a.c.k_scale : a.c.v_scale)[at]) << 23);
    store_codes_bf16((is_k ? a.wide_k : a.wide_v) + (static_cast<size_t>(p) * rows + r) * 128, l, w, sc);
  }
}

}  // namespace

cudaError_t launch_cache_widen(const SharedAttnArgs& a, cudaStream_t st) {
  const long long pages = a.prefix_len / kPage + static_cast<long long>(a.c.num_seqs) * a.wide_own;
  if (pages <= 0) return cudaSuccess;
  count_launch();
  return launch_pdl(cache_widen_kernel, dim3(static_cast<unsigned>(pages)), dim3(kReadThreads), 0, st, a);
}

cudaError_t launch_cache_append(const AppendArgs& a, bool f32, cudaStream_t st) {
  if (a.num_tokens <= 0) return cudaSuccess;
  count_launch();
  const RopeTable rt = a.theta > 0.f ? make_rope_table(a.theta) : RopeTable{};
  return f32 ? launch_pdl(cache_append_kernel<float>, dim3(a.num_tokens), dim3(kAppendThreads), 0, st, a, rt)
             : launch_pdl(cache_append_kernel<bf16>, dim3(a.num_tokens), dim3(kAppendThreads), 0, st, a, rt);
}

cudaError_t launch_cache_read(const CacheView& c, const int* seq, const int* pos, int num_tokens, bf16* k_out,
                              bf16* v_out, cudaStream_t st) {
  const long long rows = static_cast<long long>(num_tokens) * 2 * c.hkv;
  if (rows <= 0) return cudaSuccess;
  count_launch();
  return launch_pdl(cache_read_kernel, dim3(static_cast<unsigned>((rows + kReadGroups - 1) / kReadGroups)),
                    dim3(kReadThreads), 0, st, c, seq, pos, num_tokens, k_out, v_out);
}

}  // namespace quail
