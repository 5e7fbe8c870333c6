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

// A lane's 16 elements of a head row as pairs: x[0..3] = dims 8l.., x[4..7] =
// dims 64 + 8l.. ; Raw holds them as loaded.
template <typename T>
struct Raw {
  uint4 v[sizeof(T)];  // 2 x 16 bytes of bf16, 4 of fp32
  __device__ __forceinline__ void load(const T* p, int l) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)); ++i)
      v[i] = ldg_stream(p + (2 * i < static_cast<int>(sizeof(T)) ? 0 : 64) + 8 * l + (sizeof(T) == 4 ? 4 * (i & 1) : 0));
  }
  __device__ __forceinline__ void pairs(float2 (&x)[8]) const {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(v);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (sizeof(T) == 2)
        x[i] = unpack_bf16(w[i]);
      else
        x[i] = make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    }
  }
};

__device__ __forceinline__ void store_row_bf16(bf16* p, int l, const float2 (&x)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
    *reinterpret_cast<uint4*>(p + 64 * h + 8 * l) =
        make_uint4(pack_bf16(x[4 * h].x, x[4 * h].y), pack_bf16(x[4 * h + 1].x, x[4 * h + 1].y),
                   pack_bf16(x[4 * h + 2].x, x[4 * h + 2].y), pack_bf16(x[4 * h + 3].x, x[4 * h + 3].y));
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
__device__ __forceinline__ void store_row_codes(uint8_t* p, uint8_t* scale, int l, const float2 (&x)[8], float m) {
  const int e = scale_exponent(m);
  const float inv = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 a = x[4 * h + 2 * i], b = x[4 * h + 2 * i + 1];
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a.x * inv, a.y * inv), __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(b.x * inv, b.y * inv), __NV_SATFINITE, __NV_E4M3);
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

// cos and sin of pos * (w.x + w.y) for pos < 2^24, at most 1.6e-7 off (its arithmetic
// against 64 bits at every position and j for theta 1e6, 1.57e-7, and at every third for
// 1.001 and 2): what an e4m3 or bf16 rounding makes of a rotated element then differs from
// exact arithmetic's as rarely as fp32 allows. The product is held in two floats; multiples of pi/2
// (two floats) come off it in two steps, the first exactly (k * C1 is a multiple of
// 2^-23, like the product's leading float); what is left, at most pi/4, goes into the
// Taylor series, whose next terms are below 3e-8, and the trailing float into one
// step of the angle sum.
__device__ __forceinline__ void cos_sin(int pos, float2 w, float& c, float& s) {
  constexpr float kC1 = 1.57079637050628662f, kC2 = -4.37113900018624283e-8f, kInv = 0.636619772367581343f;
  const float p = static_cast<float>(pos);
  const float a = p * w.x;
  const float k = rintf(a * kInv);
  const float r = fmaf(-k, kC1, a), lo = fmaf(-k, kC2, fmaf(p, w.x, -a) + p * w.y);
  float t = r + lo;
  const float d = t - r;
  float tl = (r - (t - d)) + (lo - d);
  const float k2 = rintf(t * kInv);
  t = fmaf(-k2, kC1, t);
  tl = fmaf(-k2, kC2, tl);
  const float u = t + tl, ul = tl - (u - t), z = u * u;
  const float sp = fmaf(u * z, fmaf(z, fmaf(z, fmaf(z, 1.f / 362880.f, -1.f / 5040.f), 1.f / 120.f), -1.f / 6.f), u);
  const float cp = fmaf(z, fmaf(z, fmaf(z, fmaf(z, 1.f / 40320.f, -1.f / 720.f), 1.f / 24.f), -0.5f), 1.f);
  const float su = fmaf(cp, ul, sp), cu = fmaf(-sp, ul, cp);
  const int q = static_cast<int>(k) + static_cast<int>(k2);
  const float x = (q & 1) ? su : cu, y = (q & 1) ? cu : su;
  c = ((q + 1) & 2) ? -x : x;
  s = (q & 2) ? -y : y;
}
// 1 / sqrt(v): the hardware's value and one Newton step.
__device__ __forceinline__ float inv_sqrt(float v) {
  const float r = rsqrtf(v);
  return r > 0.f ? r * fmaf(-0.5f * v * r, r, 1.5f) : r;  // 0: the squares overflowed
}

// ------------------------------------------------------------------ append
// Block = TOK tokens: thread i first computes angle i % 64 of token i / 64 and
// looks up its page while the first rows are on their way, then 32 row groups
// of eight lanes walk the tokens' hq + 2 hkv heads, each one row ahead with its
// loads. The gains go into the token's rotation once,
//   y_j = r (x_j A_j + x_j+64 B_j),  y_j+64 = r (x_j+64 C_j + x_j D_j),  r = 1 / rms,
//   A = g_j cos, B = -g_j+64 sin, C = g_j+64 cos, D = g_j sin,
// so a row costs four products a pair and one by r: with angles and gains
// applied row by row the kernel was bound by its instructions, not by memory.
// 23,100 tokens of 48 heads, bf16 in: e4m3 cache 103 us, 5.1 TB/s, L1 at 78%; bf16 cache
// 102 us, 5.6 TB/s. The rotations kept in registers (a warp to a token) cost occupancy,
// 107 us (e4m3); two rows ahead 131, 16 tokens a block 109.
constexpr int kAppendThreads = 256;
constexpr int kAppendGroups = kAppendThreads / kRowLanes;

template <typename T, int TOK>
__global__ void __launch_bounds__(kAppendThreads) cache_append_kernel(AppendArgs a, RopeTable rt) {
  __shared__ __align__(16) float s_turn[TOK][2][4][64];  // queries, keys; A, B, C, D
  __shared__ int s_page[TOK], s_slot[TOK];               // page -1: nothing of the token is written
  grid_dependency_wait();
  grid_launch_dependents();
  const int t0 = blockIdx.x * TOK;
  const int l = threadIdx.x % kRowLanes, heads = a.hq + 2 * a.c.hkv;
  const int rows = min(TOK, a.num_tokens - t0) * heads;
  int r = threadIdx.x / kRowLanes, tok = r / heads, h = r - tok * heads;
  const T* qkv = static_cast<const T*>(a.qkv);
  Raw<T> next;
  if (r < rows) next.load(qkv + (t0 + tok) * a.ld + h * 128, l);
  if (threadIdx.x < 64 * TOK) {
    const int i = threadIdx.x / 64, j = threadIdx.x % 64, t = t0 + i;
    const int seq = t < a.num_tokens ? a.seq[t] : -1;
    const int pos = seq >= 0 ? a.pos[t] : 0;
    if (j == 0) {
      s_page[i] = seq < 0 ? -1 : page_of(a.c, seq, pos, t);
      s_slot[i] = pos % kPage;
    }
    float c = 1.f, sn = 0.f;
    if (a.theta > 0.f) cos_sin(pos, rt.w[j], c, sn);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const bf16* g = k == 0 ? a.gq : a.gk;
      const float g1 = g != nullptr ? __bfloat162float(g[j]) : 1.f;
      const float g2 = g != nullptr ? __bfloat162float(g[j + 64]) : 1.f;
      s_turn[i][k][0][j] = g1 * c;
      s_turn[i][k][1][j] = -g2 * sn;
      s_turn[i][k][2][j] = g2 * c;
      s_turn[i][k][3][j] = g1 * sn;
    }
  }
  __syncthreads();
  const int rounds = (rows + kAppendGroups - 1) / kAppendGroups;
  // whole warps take every round: the row sums shuffle over all lanes
  for (int it = 0; it < rounds; ++it) {
    const Raw<T> raw = next;
    const bool in = r < rows;
    const int ct = in ? tok : 0, ch = h;  // rows past the end index the tables of token 0, and write nothing
    r += kAppendGroups;
    h += kAppendGroups;
    while (h >= heads) {
      h -= heads;
      ++tok;
    }
    if (r < rows) next.load(qkv + (t0 + tok) * a.ld + h * 128, l);
    const int page = in ? s_page[ct] : -1;
    const bool live = page >= 0;
    const bool is_q = ch < a.hq, is_k = !is_q && ch < a.hq + a.c.hkv;
    const bool norm = is_q ? a.gq != nullptr : is_k && a.gk != nullptr;
    const bool turn = (is_q || is_k) && (norm || a.theta > 0.f);
    float2 x[8];
    raw.pairs(x);
    if (__any_sync(0xffffffffu, live && turn)) {
      float2 ss = mul2(x[0], x[0]);
#pragma unroll
      for (int i = 1; i < 8; ++i) ss = fma2(x[i], x[i], ss);
      const float f = row_sum(ss.x + ss.y);
      if (turn) {
        const float4* tab = reinterpret_cast<const float4*>(&s_turn[ct][is_q ? 0 : 1][0][8 * l]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float4 A = tab[i], B = tab[16 + i], C = tab[32 + i], D = tab[48 + i];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float2 x1 = x[2 * i + k], x2 = x[2 * i + k + 4];
            x[2 * i + k] = fma2(x1, k ? make_float2(A.z, A.w) : make_float2(A.x, A.y),
                                mul2(x2, k ? make_float2(B.z, B.w) : make_float2(B.x, B.y)));
            x[2 * i + k + 4] = fma2(x2, k ? make_float2(C.z, C.w) : make_float2(C.x, C.y),
                                    mul2(x1, k ? make_float2(D.z, D.w) : make_float2(D.x, D.y)));
          }
        }
        if (norm) {
          const float rs = inv_sqrt(f * (1.f / 128.f) + a.eps);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = mul2(x[i], make_float2(rs, rs));
        }
      }
    }
    if (live && is_q && a.q_out != nullptr)
      store_row_bf16(a.q_out + (static_cast<size_t>(t0 + ct) * a.hq + ch) * 128, l, x);
    const bool kv = live && !is_q;
    const int g = ch - a.hq - (is_k ? 0 : a.c.hkv);
    const size_t at = (static_cast<size_t>(page) * a.c.hkv + g) * kPage + s_slot[ct];
    if (!a.c.codes) {
      if (kv) store_row_bf16(static_cast<bf16*>(is_k ? a.c.k : a.c.v) + at * 128, l, x);
    } else if (__any_sync(0xffffffffu, kv)) {
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float u = fabsf(x[i].x), v = fabsf(x[i].y);
        m = fmaxf(m, fmaxf(u < INFINITY ? u : 0.f, v < INFINITY ? v : 0.f));
      }
      m = row_max(m);
      if (kv)
        store_row_codes(static_cast<uint8_t*>(is_k ? a.c.k : a.c.v) + at * 128, (is_k ? a.c.k_scale : a.c.v_scale) + at,
                        l, x, m);
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

// A lane's sixteen codes of a row (elements 8 l .. and 64 + 8 l ..), and the same
// times sc as bf16: every store of the eight lanes is a whole 128-byte line.
__device__ __forceinline__ uint4 load_codes(const uint8_t* p, int l) {
  const uint2 a = __ldcs(reinterpret_cast<const uint2*>(p + 8 * l));
  const uint2 b = __ldcs(reinterpret_cast<const uint2*>(p + 64 + 8 * l));
  return make_uint4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void store_codes_bf16(bf16* out, int l, const uint4& w, float sc) {
  const uint32_t in[4] = {w.x, w.y, w.z, w.w};
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[2 * i] = codes_to_bf16x2(in[i], sc);
    o[2 * i + 1] = codes_to_bf16x2(in[i] >> 16, sc);
  }
  __stcs(reinterpret_cast<uint4*>(out + 8 * l), make_uint4(o[0], o[1], o[2], o[3]));
  __stcs(reinterpret_cast<uint4*>(out + 64 + 8 * l), make_uint4(o[4], o[5], o[6], o[7]));
}

// Block = a few consecutive tokens: their pages are looked up once, then every
// group copies kReadRows rows at a time, loads first. 131,072 tokens of 8 heads: e4m3
// 124 us, 6.5 TB/s, 96% of a plain copy; bf16 159 us, 6.8 TB/s (five blocks an SM leave it
// 48 registers, and it spills 44 bytes).
constexpr int kReadRows = 4;
constexpr int kReadTokens = 64;  // at most

inline __host__ __device__ int read_tokens(int hkv) {  // tokens of a block: about 4 x 32 rows
  const int n = kReadRows * kReadGroups / (2 * hkv);
  return n < 1 ? 1 : n > kReadTokens ? kReadTokens : n;
}

template <bool CODES>
__global__ void __launch_bounds__(kReadThreads, 5)
    cache_read_kernel(CacheView c, const int* seq, const int* pos, int num_tokens, bf16* k_out, bf16* v_out) {
  __shared__ long long first_row[kReadTokens];  // row of the token's slot for head 0; -1: nothing to read
  grid_dependency_wait();
  grid_launch_dependents();
  const int tokens = read_tokens(c.hkv);
  const int t0 = blockIdx.x * tokens;
  if (threadIdx.x < tokens) {
    const int t = t0 + threadIdx.x;
    long long at = -1;
    if (t < num_tokens) {
      const int s = seq[t], p = pos[t];
      const int page = s < 0 ? -1 : page_of(c, s, p, t);
      if (page >= 0) at = static_cast<long long>(page) * c.hkv * kPage + p % kPage;
    }
    first_row[threadIdx.x] = at;
  }
  __syncthreads();
  const int l = threadIdx.x % kRowLanes, per = 2 * c.hkv, rows = tokens * per;
  for (int r0 = threadIdx.x / kRowLanes; r0 < rows; r0 += kReadRows * kReadGroups) {
    uint4 x[kReadRows][CODES ? 1 : 2];
    float sc[kReadRows];
    bf16* out[kReadRows];
#pragma unroll
    for (int k = 0; k < kReadRows; ++k) {
      const int r = r0 + k * kReadGroups;
      const int t = r / per, kvh = r - t * per;
      const bool is_k = kvh < c.hkv;
      const int h = is_k ? kvh : kvh - c.hkv;
      out[k] = is_k ? k_out : v_out;
      if (r >= rows || first_row[r < rows ? t : 0] < 0) out[k] = nullptr;
      if (out[k] == nullptr) continue;
      out[k] += (static_cast<size_t>(t0 + t) * c.hkv + h) * 128;
      const size_t at = static_cast<size_t>(first_row[t]) + static_cast<size_t>(h) * kPage;
      if constexpr (CODES) {
        x[k][0] = load_codes(static_cast<const uint8_t*>(is_k ? c.k : c.v) + at * 128, l);
        sc[k] = __uint_as_float(static_cast<uint32_t>((is_k ? c.k_scale : c.v_scale)[at]) << 23);
      } else {
        const bf16* in = static_cast<const bf16*>(is_k ? c.k : c.v) + at * 128;
        x[k][0] = ldg_stream(in + 8 * l);
        x[k][1] = ldg_stream(in + 64 + 8 * l);
      }
    }
#pragma unroll
    for (int k = 0; k < kReadRows; ++k) {
      if (out[k] == nullptr) continue;
      if constexpr (CODES) {
        store_codes_bf16(out[k], l, x[k][0], sc[k]);
      } else {
        __stcs(reinterpret_cast<uint4*>(out[k] + 8 * l), x[k][0]);
        __stcs(reinterpret_cast<uint4*>(out[k] + 64 + 8 * l), x[k][1]);
      }
    }
  }
}

// ------------------------------------------------------------------ answer token
// The answer token of a letters call: one normed row q | k | v for all documents.
// answer_query_kernel turns its q by each document's length; answer_join_kernel
// adds its own key and value to what the document gave. Score and value of the
// own key stay fp32 and never pass through the cache: q and k are turned by the
// same angle, so q . k is the unturned rows' product, and with the document's
// (o, lse),  o' = (o e^lse + v e^s) / (e^lse + e^s),  s = q . k / sqrt(128).
// A few MB at most for thousands of documents: latency is what they cost.
__global__ void __launch_bounds__(256) answer_query_kernel(const float* qkv, const int* len, int hq, bf16* q,
                                                           RopeTable rt) {
  __shared__ float2 s_cs[64];
  grid_dependency_wait();
  if (threadIdx.x < 64) cos_sin(len[blockIdx.x], rt.w[threadIdx.x], s_cs[threadIdx.x].x, s_cs[threadIdx.x].y);
  __syncthreads();
  bf16* out = q + static_cast<size_t>(blockIdx.x) * hq * 128;
  for (int i = threadIdx.x; i < hq * 32; i += 256) {  // two neighbouring pairs (j, j + 64)
    const int h = i / 32, j = i % 32 * 2;
    const float2 x = *reinterpret_cast<const float2*>(qkv + h * 128 + j);
    const float2 y = *reinterpret_cast<const float2*>(qkv + h * 128 + 64 + j);
    const float2 t0 = s_cs[j], t1 = s_cs[j + 1];
    uint32_t* o = reinterpret_cast<uint32_t*>(out + h * 128 + j);
    o[0] = pack_bf16(x.x * t0.x - y.x * t0.y, x.y * t1.x - y.y * t1.y);
    o[32] = pack_bf16(y.x * t0.x + x.x * t0.y, y.y * t1.x + x.y * t1.y);
  }
}

// A warp per (document, head); out rows are the two-term splits that W_o reads.
__global__ void __launch_bounds__(256) answer_join_kernel(const float* qkv, const bf16* o, const float* lse, int rows,
                                                          int hq, int group, bf16* out) {
  grid_dependency_wait();
  const int r = blockIdx.x * 8 + threadIdx.x / 32, lane = threadIdx.x % 32;
  if (r >= rows) return;
  const int doc = r / hq, h = r % hq, kv = h / group;
  const float4 x = *reinterpret_cast<const float4*>(qkv + h * 128 + 4 * lane);
  const float4 k = *reinterpret_cast<const float4*>(qkv + (hq + kv) * 128 + 4 * lane);
  const float4 v = *reinterpret_cast<const float4*>(qkv + (hq + hq / group + kv) * 128 + 4 * lane);
  float s = x.x * k.x + x.y * k.y + x.z * k.z + x.w * k.w;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  s *= 0.08838834764831845f;
  const float le = lse[r], m = fmaxf(le, s);
  const float wd = __expf(le - m), ws = __expf(s - m);  // an empty document: lse = -inf, weight 0
  const float inv = 1.f / (wd + ws), a = wd * inv, b = ws * inv;
  const uint2 od = *reinterpret_cast<const uint2*>(o + static_cast<size_t>(r) * 128 + 4 * lane);
  const float2 d0 = unpack_bf16(od.x), d1 = unpack_bf16(od.y);
  uint2 hi, lo;
  split_bf16(a * d0.x + b * v.x, a * d0.y + b * v.y, hi.x, lo.x);
  split_bf16(a * d1.x + b * v.z, a * d1.y + b * v.w, hi.y, lo.y);
  bf16* row = out + static_cast<size_t>(doc) * 2 * hq * 128 + h * 128 + 4 * lane;
  *reinterpret_cast<uint2*>(row) = hi;
  *reinterpret_cast<uint2*>(row + hq * 128) = lo;
}

// theta^(-2j/128) for all j from one power: in 64 bits the products are off by up to
// 2^-47 (j times the power's rounding and a product's; measured 2^-47.8), a little more than
// the 2^-49 that two floats hold; cos_sin's bound includes it. 64 powers a call took the
// host longer than the launch.
RopeTable angle_table(float theta) {
  RopeTable t;
  const double step = std::pow(static_cast<double>(theta), -1.0 / 64.0);
  double w = 1.0;
  for (float2& x : t.w) {
    x.x = static_cast<float>(w);
    x.y = static_cast<float>(w - static_cast<double>(x.x));
    w *= step;
  }
  return t;
}

}  // namespace

cudaError_t launch_answer_query(const float* qkv, const int* len, int n, int hq, float theta, bf16* q, cudaStream_t st) {
  count_launch();
  return launch_pdl(answer_query_kernel, dim3(n), dim3(256), 0, st, qkv, len, hq, q, angle_table(theta));
}

cudaError_t launch_answer_join(const float* qkv, const bf16* o, const float* lse, int n, int hq, int hkv, bf16* out,
                               cudaStream_t st) {
  count_launch();
  return launch_pdl(answer_join_kernel, dim3((n * hq + 7) / 8), dim3(256), 0, st, qkv, o, lse, n * hq, hq, hq / hkv, out);
}

namespace {

template <typename T>
cudaError_t launch_append(const AppendArgs& a, int num_sms, cudaStream_t st) {
  const RopeTable rt = a.theta > 0.f ? angle_table(a.theta) : RopeTable{};
  // Few tokens: a block each, so that they spread over the SMs. One / four a block, us:
  // 4 tokens 3.2 / 5.5, 256 3.9 / 5.7, 608 5.0 / 5.8, 800 7.7 / 7.4, 1,216 8.7 / 7.6
  // (48 heads, bf16; e4m3 9.8 / 10.1 at 608, 12.7 / 11.7 at 800).
  if (a.num_tokens <= 4 * num_sms)
    return launch_pdl(cache_append_kernel<T, 1>, dim3(a.num_tokens), dim3(kAppendThreads), 0, st, a, rt);
  return launch_pdl(cache_append_kernel<T, 4>, dim3((a.num_tokens - 1) / 4 + 1), dim3(kAppendThreads), 0, st, a, rt);
}

}  // namespace

cudaError_t launch_cache_append(const AppendArgs& a, bool f32, int num_sms, cudaStream_t st) {
  if (a.num_tokens <= 0) return cudaSuccess;
  count_launch();
  return f32 ? launch_append<float>(a, num_sms, st) : launch_append<bf16>(a, num_sms, st);
}

cudaError_t launch_cache_read(const CacheView& c, const int* seq, const int* pos, int num_tokens, bf16* k_out,
                              bf16* v_out, cudaStream_t st) {
  if (num_tokens <= 0) return cudaSuccess;
  const int tokens = read_tokens(c.hkv);
  const dim3 grid(static_cast<unsigned>((num_tokens + static_cast<long long>(tokens) - 1) / tokens));
  count_launch();
  return c.codes ? launch_pdl(cache_read_kernel<true>, grid, dim3(kReadThreads), 0, st, c, seq, pos, num_tokens, k_out, v_out)
                 : launch_pdl(cache_read_kernel<false>, grid, dim3(kReadThreads), 0, st, c, seq, pos, num_tokens, k_out, v_out);
}

}  // namespace quail
