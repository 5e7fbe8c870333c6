// Attention over the paged document cache for a batch whose sequences share
// their first prefix_len tokens:
//   o = softmax(scale q K^T) V,  lse = log sum exp(scale q K^T)
// The keys of a row are cut into parts (the shared prefix, pieces of the
// sequence's own pages); each part keeps (max, sum, sum of weighted values)
// and the join rescales them to one maximum.
#include <atomic>

#include "attn_common.cuh"
#include "cache_attn.cuh"
#include "launch.cuh"
#include "quail_internal.h"
#include "sm103.cuh"

namespace quail {

namespace {

// ------------------------------------------------------------------ streaming kernel
// Few query rows per KV head (a decoded token: G of them), so the work is
// reading keys and values once: every warp of the grid is a worker of its own
// with a private ring of pages, and the work list (all pages of all sequences
// and KV heads, in order) is cut into equal contiguous chunks, one per worker,
// whatever the lengths are. A worker's lanes copy a page two stages ahead, across
// the borders of work items, so the stream of loads never drains; no barrier joins
// warps. (16-byte copies by the lanes, whose arrivals complete a stage, take 0.3 to
// 1.6% less time than bulk copies of 2 KB.) Pieces of an item that several workers
// share are joined by the second kernel.
//
// Per page of 16 keys (two e4m3 pages at a time, so that the bookkeeping and the
// row reductions are shared by 32 keys), on mma.sync m16n8k16 with the query
// rows as N: S^T = K Q^T (M 16 keys, N 8 rows) and O^T += V^T P^T (M 16 dims, N 8
// rows). Keys and values are the A operands, so a few query rows waste little:
// with the rows as M, 12 of 16 rows of a 4-head group were padding, in O's
// registers, the exponentials and the products alike. A sequence with more than 8
// rows is several items in a row, so its pages come from L2 after the first (items
// of 16 rows were slower: 8 workers an SM for their registers).
// Over bf16 pages q is bf16 and P two bf16 terms, 15 bits: the products are a small part of
// the time (256 sequences behind 2,048: 126.1 us, with one term, rounded, 125.4), and o's
// error is that of its own rounding, 0.00166 relative (0.0023 with one term). Over e4m3 pages
// the codes widen exactly to fp16, q is scaled by a power of two per row (exact) and P is
// rounded to fp16, 11 bits (error 0.00167).
// The key's power of two multiplies its score, the value's is added to the
// exponent of its weight: o and l keep separate maxima, so that value rows of any
// scale neither overflow P nor starve the sum.
//
// Bound, with up to 8 rows, by HBM: 64 sequences of 2,048 own keys (8 KV heads, bf16)
// take 91 us, 5.9 TB/s; e4m3, 4,096 keys, 95 us, 5.9 TB/s. With more rows by the
// latency of its products and softmax, three workers to a scheduler: 160 clocks of an
// SM for a pass of 8 rows over an e4m3 page. Taking the units' maxima only when some
// weight would pass 2^8, without their shuffles, was 2% slower.
template <bool CODES>
struct StreamCfg {
  static constexpr int kWarps = kStreamWarps;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kUnit = stream_unit_pages(CODES);   // pages a stage
  static constexpr uint32_t kPlane = CODES ? 2048 : 4096;  // K or V of one (page, head)
  static constexpr uint32_t kStage = 2 * kPlane * kUnit;
  static constexpr int kStages = 2;
  static constexpr int kScaleLanes = CODES ? 2 * kUnit : 0;  // lanes that copy 16 scale bytes each
  static constexpr uint32_t kRing = kWarps * kStages * kStage;
  static constexpr uint32_t kScales = CODES ? kWarps * kStages * kUnit * 32 : 0;  // key, value exponents
  static constexpr uint32_t kBars = kWarps * kStages * 8;
  static constexpr uint32_t kScan = (kThreads + 1) * 8;
  static constexpr size_t kSmem = 1024 + kRing + kScales + kBars + kScan + 16;
  static_assert(kSmem <= 227 * 1024, "shared memory");
};
constexpr int kMinChunk = 2;  // units a worker takes at least
// fp16 weights are taken times 2^7: at most 2^15 with the 2^8 that a score may pass the
// reference maximum by. They keep their 11 bits down to 2^-21 of the largest, and are
// lost below 2^-32 (2^-14 and 2^-25 as they are, which a sum over 100,000 keys would show).
constexpr float kLift = 7.f;

__device__ __forceinline__ uint32_t swz(uint32_t r, uint32_t c) { return r * 128u + ((c ^ (r & 7u)) << 4); }

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint4& a, const uint2& b) {
  if constexpr (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y));
}
// Transposes an 8x8 matrix of 16-bit elements: from (row lane / 4, columns
// 2 (lane % 4) and the next) to (column lane / 4, rows 2 (lane % 4) and the next).
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// A unit of the work list (a stage: UNIT pages, fewer at an item's end): unit j
// of the n of an item. Items: (row tile, head) over the prefix, then (sequence,
// head) over own pages.
struct Cursor {
  bool own;
  int b;        // sequence, or row tile of the whole batch
  int x, X;     // item: x = head * tiles + row tile of the sequence (prefix: the head), of X
  int j, n;
};

template <int UNIT>
__device__ __forceinline__ int own_units(const SharedAttnArgs& a, int b) {
  return (own_pages(a, b) + UNIT - 1) / UNIT;
}
// Items of sequence b: its row tiles for every KV head.
__device__ __forceinline__ int own_items(const SharedAttnArgs& a, int b) {
  const int n = a.q_offsets ? a.q_offsets[b + 1] - a.q_offsets[b] : 1;
  return (n * (a.hq / a.c.hkv) + kItemRows - 1) / kItemRows * a.c.hkv;
}
// All units of sequence b; b may lie past the last.
template <int UNIT>
__device__ __forceinline__ long long seq_units(const SharedAttnArgs& a, int b, int* n) {
  *n = b < a.c.num_seqs ? own_units<UNIT>(a, b) : 0;
  return *n > 0 ? static_cast<long long>(*n) * own_items(a, b) : 0;
}
// First sequence at or after b with own pages; num_seqs if none.
template <int UNIT>
__device__ __forceinline__ void seek_own(const SharedAttnArgs& a, Cursor& c, int b, int lane) {
  c.own = true;
  c.x = c.j = 0;
  for (; b < a.c.num_seqs; b += 32) {
    const int n = b + lane < a.c.num_seqs ? own_units<UNIT>(a, b + lane) : 0;
    const uint32_t some = __ballot_sync(0xffffffffu, n > 0);
    if (some != 0) {
      const int first = __ffs(some) - 1;
      c.b = b + first;
      c.n = __shfl_sync(0xffffffffu, n, first);
      c.X = own_items(a, c.b);
      return;
    }
  }
  c.b = a.c.num_seqs;
  c.n = c.X = 0;
}
template <int UNIT>
__device__ __forceinline__ void next_unit(const SharedAttnArgs& a, Cursor& c, int lane) {
  if (++c.j < c.n) return;
  c.j = 0;
  if (++c.x < c.X) return;
  c.x = 0;
  if (c.own) {
    seek_own<UNIT>(a, c, c.b + 1, lane);
  } else if (++c.b >= a.prefix_row_tiles) {
    seek_own<UNIT>(a, c, 0, lane);
  }
}
// KV head of the cursor's item.
__device__ __forceinline__ int item_head(const SharedAttnArgs& a, const Cursor& c) {
  return c.own ? c.x / (c.X / a.c.hkv) : c.x;
}

template <bool CODES>
__global__ void __launch_bounds__(StreamCfg<CODES>::kThreads, 1)
    attention_stream_kernel(SharedAttnArgs a) {
  using Cfg = StreamCfg<CODES>;
  constexpr int kStages = Cfg::kStages, kUnit = Cfg::kUnit, kThreads = Cfg::kThreads, kRows = kItemRows;
  constexpr int kKeys = kUnit * kPage;  // keys of a unit
  extern __shared__ uint8_t smem_raw[];
  // by an offset: from an address rounded up, the compiler could not tell shared memory
  uint8_t* base = smem_raw + (-smem_u32(smem_raw) & 1023u);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* ring = base + warp * kStages * Cfg::kStage;
  uint8_t* scales = base + Cfg::kRing + warp * kStages * kUnit * 32;
  uint64_t* bars = reinterpret_cast<uint64_t*>(base + Cfg::kRing + Cfg::kScales) + warp * kStages;
  long long* scan = reinterpret_cast<long long*>(base + Cfg::kRing + Cfg::kScales + Cfg::kBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(base + Cfg::kRing + Cfg::kScales + Cfg::kBars +
                                                             Cfg::kScan);
  const long long limit_clk = pipeline_wait_limit();
  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(&bars[s], 32 + (limit_clk < 0));
    fence_mbar_init();
    if (warp == 0) *abort_flag = 0;
  }
  grid_dependency_wait();
  grid_launch_dependents();

  // ---- the plan: thread i counts the units of its own run of sequences
  const int B = a.c.num_seqs, G = a.hq / a.c.hkv;
  const int per = (B + kThreads - 1) / kThreads;
  const int b0 = min(B, static_cast<int>(threadIdx.x) * per), b1 = min(B, b0 + per);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) {
    if (blockIdx.x == 0 && !query_range(a, b).ok) raise_device_error(a.c.err, QUAIL_ERR_DEVICE_BOUNDS, b);
    int n;
    mine += seq_units<kUnit>(a, b, &n);
  }
  const int pp = a.prefix_len / kPage, pu = (pp + kUnit - 1) / kUnit;
  const long long prefix_units = static_cast<long long>(a.prefix_row_tiles) * a.c.hkv * pu;
  {
    long long x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    scan[threadIdx.x + 1] = x;  // inclusive within the warp
    if (threadIdx.x == 0) scan[0] = 0;
    __syncthreads();
    long long before = 0;
    for (int w = 0; w < warp; ++w) before += scan[32 * w + 32];
    __syncthreads();
    scan[threadIdx.x + 1] = x + before;
    __syncthreads();
  }
  const long long units = prefix_units + scan[kThreads];
  const long long workers = static_cast<long long>(gridDim.x) * Cfg::kWarps;
  const long long chunk = max(static_cast<long long>(kMinChunk), (units + workers - 1) / workers);
  if (blockIdx.x == 0) {
    long long at = prefix_units + scan[threadIdx.x];
    for (int b = b0; b < b1; ++b) {
      a.plan[2 + b] = at;
      int n;
      at += seq_units<kUnit>(a, b, &n);
    }
    if (threadIdx.x == 0) {
      a.plan[0] = units;
      a.plan[1] = chunk;
      a.plan[2 + B] = units;
    }
  }
  // workers of one SM sit far apart in the list, so long items spread over the SMs
  const long long worker = static_cast<long long>(warp) * gridDim.x + blockIdx.x;
  const long long u0 = worker * chunk;
  const int count = static_cast<int>(max(0LL, min(units, u0 + chunk) - u0));
  if (count == 0) return;

  // ---- where the chunk begins
  Cursor cc;
  if (u0 < prefix_units) {
    const long long item = u0 / pu;
    cc.own = false;
    cc.b = static_cast<int>(item / a.c.hkv);
    cc.x = static_cast<int>(item % a.c.hkv);
    cc.X = a.c.hkv;
    cc.j = static_cast<int>(u0 % pu);
    cc.n = pu;
  } else {
    const long long v = u0 - prefix_units;
    int lo = 0, hi = kThreads;  // scan[lo] <= v < scan[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (scan[mid] <= v)
        lo = mid;
      else
        hi = mid;
    }
    long long at = scan[lo];
    for (int b = lo * per;; b += 32) {
      int n;
      long long x = seq_units<kUnit>(a, b + lane, &n);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, at + x > v);
      if (past != 0) {
        const int f = __ffs(past) - 1;
        const long long end = __shfl_sync(0xffffffffu, at + x, f);
        cc.own = true;
        cc.b = b + f;
        cc.n = __shfl_sync(0xffffffffu, n, f);
        cc.X = own_items(a, cc.b);
        const long long rem = v - (end - static_cast<long long>(cc.n) * cc.X);
        cc.x = static_cast<int>(rem / cc.n);
        cc.j = static_cast<int>(rem % cc.n);
        break;
      }
      at = __shfl_sync(0xffffffffu, at + x, 31);
      if (b >= B) return;  // not reached: v lies before the end of the list
    }
  }

  // ---- producer: unit `issued` of the chunk into stage issued % kStages. Page
  // ids are read 32 at a time, one per lane, while the units before are at work.
  Cursor pc = cc;
  int issued = 0, win = 0, ids = 0, pages = 0, head = 0;  // ids: pages win .. win + 31 of the item's `pages`
  const int* list = nullptr;
  auto open_list = [&]() {
    list = pc.own ? a.c.table + static_cast<size_t>(pc.b) * a.c.max_pages + pp : a.prefix_pages;
    pages = pc.own ? own_pages(a, pc.b) : pp;
    head = item_head(a, pc);
    win = pc.j * kUnit;
    ids = win + lane < pages ? list[win + lane] : -1;
  };
  if (pc.n > 0) open_list();
  // the lane's 16-byte chunk of rows lane / 8 + 4 k of a plane (or half of one)
  const uint32_t from = (lane >> 3) * (CODES ? 128 : 256) + (lane & 7) * 16;
  const uint32_t to[2] = {swz(lane >> 3, lane & 7), swz(4 + (lane >> 3), lane & 7) - 512};
  auto produce = [&]() {
    const int j0 = pc.j * kUnit;
    const int s = issued % kStages;
    int page[kUnit];
    bool bad = false;
#pragma unroll
    for (int u = 0; u < kUnit; ++u) {
      page[u] = __shfl_sync(0xffffffffu, ids, j0 - win + u);
      const bool ok = page[u] >= 0 && page[u] < a.c.num_pages;
      bad = bad || (!ok && j0 + u < pages);
      if (!ok) page[u] = -1;
    }
    if (bad && lane == 0) raise_device_error(a.c.err, QUAIL_ERR_DEVICE_BOUNDS, pc.own ? pc.b : 0);
#pragma unroll
    for (int u = 0; u < kUnit; ++u) {
      if (page[u] < 0) continue;  // the stage's old contents are consumed; the rows are void
      const size_t row = static_cast<size_t>(page[u] * a.c.hkv + head) * kPage;
      const uint32_t dst = smem_u32(ring + s * Cfg::kStage + u * 2 * Cfg::kPlane);
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const uint8_t* src = static_cast<const uint8_t*>(kv == 0 ? a.c.k : a.c.v) + row * (CODES ? 128 : 256) + from;
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int h = 0; h < (CODES ? 1 : 2); ++h)
            copy16_async(dst + kv * Cfg::kPlane + h * 2048 + k * 512 + to[k & 1], src + k * (CODES ? 512 : 1024) + h * 128);
      }
    }
    if (CODES && lane < Cfg::kScaleLanes) {  // lane 2u: the keys' exponents of page u, 2u + 1: the values'
      const int p = lane < 2 ? page[0] : page[kUnit - 1];
      if (p >= 0)
        copy16_async(smem_u32(scales + s * kUnit * 32 + lane * 16),
                     ((lane & 1) ? a.c.v_scale : a.c.k_scale) + static_cast<size_t>(p * a.c.hkv + head) * kPage);
    }
    arrive_after_copies(&bars[s]);
    ++issued;
    if (issued == count) return;
    const int j = pc.j;
    next_unit<kUnit>(a, pc, lane);
    if (pc.j != j + 1) {
      open_list();
    } else if (pc.j * kUnit - win >= 32) {
      win += 32;
      ids = win + lane < pages ? list[win + lane] : -1;
    }
  };
  for (int s = 0; s < kStages && s < count; ++s) produce();

  // ---- consumer
  const int gq = lane >> 2, tq = lane & 3;
  // The 16 keys of a page go to the two halves of M so that lane group gq's two
  // accumulator rows are keys 2 gq and 2 gq + 1 (their exponents one half word)
  // and the 8 keys of a half fall on eight different swizzle positions: row i
  // of half t is key 2 i + (t ^ (i >> 2)).
  auto half_key = [](int t, int i) { return 2 * i + (t ^ (i >> 2)); };
  const int my_key[2] = {half_key(0, gq), half_key(1, gq)};
  // ldmatrix offsets within a plane (or half of one): lane 8 i + j addresses row
  // j of matrix i: (half 0, chunk 2 c), (1, 2 c), (0, 2 c + 1), (1, 2 c + 1).
  uint32_t off[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) off[c] = swz(half_key((lane >> 3) & 1, lane & 7), 2 * c + (lane >> 4));

  uint2 qf[8];     // Q^T fragments
  float o[8][4];   // O^T: 16 dims x 8 rows
  float2 m_o, m_l, l, f_row;  // of rows 2 tq, 2 tq + 1; l: this lane's keys only
  int limit[2];    // keys that those rows see, counted from the item's first
  QueryRange qr{0, 0, 0, true};
  int g = 0, flat0 = 0, n_rows = 0;  // KV head, first row (within the sequence or the batch), rows
  int first_unit = 0;
  int keys = 0, safe = 0;  // the item's keys; those that every row sees
  bool ok = true;

  // the item's query rows: fragments, score factors, limits; an empty state
  auto open_item = [&]() {
    g = item_head(a, cc);
    if (cc.own) {
      qr = query_range(a, cc.b);
      flat0 = cc.x % (cc.X / a.c.hkv) * kRows;
      n_rows = min(kRows, (qr.hi - qr.lo) * G - flat0);
      keys = qr.len - a.prefix_len;
      safe = a.causal ? keys - (qr.hi - qr.lo - 1) + flat0 / G : keys;
    } else {
      qr.lo = 0;
      flat0 = cc.b * kRows;
      n_rows = min(kRows, a.total_q * G - flat0);
      keys = safe = a.prefix_len;
    }
    first_unit = cc.j;
    // fragment of 16 dims: row gq, the dims that lane tq's A registers hold
    const int flat = flat0 + gq;
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) qf[ks] = make_uint2(0u, 0u);
    if (gq < n_rows) {
      const uint32_t* p = reinterpret_cast<const uint32_t*>(
          a.q + (static_cast<size_t>(qr.lo + flat / G) * a.hq + g * G + flat % G) * 128);
#pragma unroll
      for (int ks = 0; ks < 8; ++ks)
        qf[ks] = CODES ? *reinterpret_cast<const uint2*>(p + ks * 8 + 2 * tq)
                       : make_uint2(p[ks * 8 + tq], p[ks * 8 + tq + 4]);
    }
    f_row = make_float2(a.scale_log2, a.scale_log2);
    if constexpr (CODES) {
      float am = 0.f;
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        const float2 x = unpack_bf16(qf[ks].x), y = unpack_bf16(qf[ks].y);
        am = fmaxf(fmaxf(fmaxf(am, fabsf(x.x)), fmaxf(fabsf(x.y), fabsf(y.x))), fabsf(y.y));
      }
      am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 1));
      am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 2));
      // 2^e <= max |q| < 2^(e+1), e in [-126, 126]: q / 2^e is exact in fp16
      // down to 2^-24 of the row's maximum
      const int e = am > 0.f ? min(126, max(-126, static_cast<int>(__float_as_uint(am) >> 23) - 127)) : 0;
      const float down = pow2_byte(127 - e), f = a.scale_log2 * pow2_byte(127 + e);
      f_row = make_float2(__shfl_sync(0xffffffffu, f, 8 * tq), __shfl_sync(0xffffffffu, f, 8 * tq + 4));
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        const float2 x = unpack_bf16(qf[ks].x), y = unpack_bf16(qf[ks].y);
        qf[ks] = make_uint2(pack_f16(x.x * down, x.y * down), pack_f16(y.x * down, y.y * down));
      }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int rc = 2 * tq + e;
      limit[e] = cc.own && a.causal && rc < n_rows ? keys - (qr.hi - qr.lo - 1 - (flat0 + rc) / G) : keys;
    }
    m_o = m_l = make_float2(-INFINITY, -INFINITY);
    l = make_float2(0.f, 0.f);
#pragma unroll
    for (int n = 0; n < 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
  };

  // the piece's rows: final when it is the whole of what they attend to, else parts
  auto close_item = [&]() {
    const bool whole = cc.own && a.prefix_len == 0 && first_unit == 0 && cc.j == cc.n - 1;
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) {
      l.x += __shfl_xor_sync(0xffffffffu, l.x, x);
      l.y += __shfl_xor_sync(0xffffffffu, l.y, x);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = 2 * tq + e;
      const float sum = e ? l.y : l.x, ml = e ? m_l.y : m_l.x;
      const float mo = (e ? m_o.y : m_o.x) - (CODES ? 127.f + kLift : 0.f);
      const int flat = flat0 + min(r, n_rows - 1);
      const size_t row = static_cast<size_t>(qr.lo + flat / G) * a.hq + g * G + flat % G;
      const bool rest = first_unit > 0;  // the piece continues an earlier worker's
      const size_t at = rest ? static_cast<size_t>(worker) * kRows + r : row;
      float* po = rest ? a.cont_o : cc.own ? a.own_o : a.prefix_o;
      PartStat* ps = rest ? a.cont_st : cc.own ? a.own_st : a.prefix_st;
      // 2^(m_o - m_l) brings values summed at m_o to the weights' maximum
      const float f = whole ? (CODES ? exp2f(mo - ml) : 1.f) / sum : 1.f;
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        // two neighbouring dims of the 16 per lane: e4m3 products leave them so, bf16
        // ones trade with the neighbour (dims gq and gq + 8 -> a pair of one half)
        float v0 = o[n][e], v1 = o[n][2 + e];
        int dim = 16 * n + 2 * gq;
        if constexpr (!CODES) {
          const bool odd = gq & 1;
          const float got = __shfl_xor_sync(0xffffffffu, odd ? v0 : v1, 4);
          (odd ? v0 : v1) = got;
          dim = 16 * n + (odd ? 8 : 0) + (gq & ~1);
        }
        if (r < n_rows) {
          if (whole)
            *reinterpret_cast<uint32_t*>(a.out + row * 128 + dim) = pack_bf16(v0 * f, v1 * f);
          else
            *reinterpret_cast<float2*>(po + at * 128 + dim) = make_float2(v0, v1);
        }
      }
      if (gq == 0 && r < n_rows) {
        if (!whole)
          ps[at] = PartStat{mo, ml, sum, 0.f};
        else if (a.lse != nullptr)
          a.lse[row] = (ml + log2f(sum)) * 0.6931471805599453f;
      }
    }
  };

  for (int i = 0; i < count; ++i) {
    const int s = i % kStages;
    if (i == 0 || cc.j == 0) open_item();
    // warp-uniform wait: the collectives below need every lane
    if (!__all_sync(0xffffffffu, wait_bar(&bars[s], static_cast<uint32_t>((i / kStages) & 1), abort_flag, limit_clk))) {
      ok = false;
      break;
    }
    const uint32_t stage = smem_u32(ring + s * Cfg::kStage);
    const int key0 = cc.j * kKeys;
    const bool border = key0 + kKeys > safe;  // some row does not see some key of the unit
    float2 sc[2 * kUnit];  // scores of this lane's keys (half 0, half 1 of each page), its two rows
    {
      float acc[kUnit][2][4] = {};  // two chains, for independent products
#pragma unroll
      for (int u = 0; u < kUnit; ++u) {
        const uint32_t kb = stage + u * 2 * Cfg::kPlane;
#pragma unroll
        for (int c = 0; c < (CODES ? 4 : 8); ++c) {
          uint32_t r[4];  // halves 0 and 1 of one chunk, then of the next
          ldsm_x4(kb + (CODES ? 0 : (c >> 2) * 2048) + off[c & 3], r);
          if constexpr (CODES) {  // a chunk is 16 dims
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint4 A;
              widen4(r[2 * h], A.x, A.z);
              widen4(r[2 * h + 1], A.y, A.w);
              mma16816<true>(acc[u][h], A, qf[2 * c + h]);
            }
          } else {
            const uint4 A = make_uint4(r[0], r[1], r[2], r[3]);
            mma16816<false>(acc[u][c & 1], A, qf[c]);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kUnit; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          sc[2 * u + h] = add2(make_float2(acc[u][0][2 * h], acc[u][0][2 * h + 1]),
                              make_float2(acc[u][1][2 * h], acc[u][1][2 * h + 1]));
    }
    float ve[2 * kUnit];  // value exponents of this lane's keys, biased by 127
#pragma unroll
    for (int k = 0; k < 2 * kUnit; ++k) {
      float kf = 1.f;
      if constexpr (CODES) {
        const uint8_t* e = scales + (s * kUnit + (k >> 1)) * 32 + my_key[k & 1];
        kf = pow2_byte(e[0]);
        // byte b as the float 2^23 + b, exactly
        ve[k] = __uint_as_float(0x4b000000u | e[16]) - 8388608.f;
      }
      sc[k] = mul2(sc[k], CODES ? mul2(f_row, make_float2(kf, kf)) : f_row);
    }
    if (border) {
#pragma unroll
      for (int k = 0; k < 2 * kUnit; ++k) {
        const int key = key0 + (k >> 1) * kPage + my_key[k & 1];
        if (key >= limit[0]) sc[k].x = -INFINITY;
        if (key >= limit[1]) sc[k].y = -INFINITY;
      }
    }
    float2 ml = sc[0];
#pragma unroll
    for (int k = 1; k < 2 * kUnit; ++k) ml = make_float2(fmaxf(ml.x, sc[k].x), fmaxf(ml.y, sc[k].y));
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) {
      ml.x = fmaxf(ml.x, __shfl_xor_sync(0xffffffffu, ml.x, x));
      ml.y = fmaxf(ml.y, __shfl_xor_sync(0xffffffffu, ml.y, x));
    }
    float2 mo = ml;
    if constexpr (CODES) {
      mo = add2(sc[0], make_float2(ve[0], ve[0]));
#pragma unroll
      for (int k = 1; k < 2 * kUnit; ++k) {
        const float2 v = add2(sc[k], make_float2(ve[k], ve[k]));
        mo = make_float2(fmaxf(mo.x, v.x), fmaxf(mo.y, v.y));
      }
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) {
        mo.x = fmaxf(mo.x, __shfl_xor_sync(0xffffffffu, mo.x, x));
        mo.y = fmaxf(mo.y, __shfl_xor_sync(0xffffffffu, mo.y, x));
      }
    }
    const bool grows = ml.x > m_l.x + 8.f || ml.y > m_l.y + 8.f || mo.x > m_o.x + 8.f || mo.y > m_o.y + 8.f;
    // The reference maxima move only when a unit exceeds them by more than
    // 2^8: weights stay below 256 and the rescale is skipped on most units.
    if (__any_sync(0xffffffffu, grows)) {
      auto step = [](float m, float n) { return n == -INFINITY ? 1.f : exp2f(m - n); };
      const float2 no = make_float2(fmaxf(m_o.x, mo.x), fmaxf(m_o.y, mo.y));
      const float2 nl = make_float2(fmaxf(m_l.x, ml.x), fmaxf(m_l.y, ml.y));
      const float2 fo = make_float2(step(m_o.x, no.x), step(m_o.y, no.y));
      l = mul2(l, make_float2(step(m_l.x, nl.x), step(m_l.y, nl.y)));
      m_o = no;
      m_l = nl;
#pragma unroll
      for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[n][c] *= (c & 1) ? fo.y : fo.x;
    }
    uint2 pb[kUnit], pl[kUnit];  // P^T fragments; over bf16 pages what their rounding left, as bf16 again
    // no key seen yet: the reference is still -inf, and every weight is 0
    auto neg = [](float m) { return m == -INFINITY ? 0.f : -m; };
    const float2 rl = make_float2(neg(m_l.x), neg(m_l.y));
    const float2 ro = make_float2(neg(m_o.x) + kLift, neg(m_o.y) + kLift);  // e4m3 only
#pragma unroll
    for (int k = 0; k < 2 * kUnit; ++k) {
      const float2 x = add2(sc[k], rl);
      const float2 e = make_float2(fast_exp2(x.x), fast_exp2(x.y));
      l = add2(l, e);
      uint32_t p;
      if constexpr (CODES) {
        const float2 v = add2(sc[k], add2(ro, make_float2(ve[k], ve[k])));
        p = pack_f16(fast_exp2(v.x), fast_exp2(v.y));
      } else {
        // the high term cut off, not rounded, and the low one not 0 beside it: an infinite
        // value times both is that infinity, not a NaN
        const uint32_t ux = __float_as_uint(e.x), uy = __float_as_uint(e.y);
        p = __byte_perm(ux, uy, 0x7632);
        const float2 h = make_float2(__uint_as_float(ux & 0xffff0000u), __uint_as_float(uy & 0xffff0000u));
        const float2 rest = fma2(h, make_float2(-1.f, -1.f), e), least = mul2(h, make_float2(0x1p-30f, 0x1p-30f));
        const uint32_t lo = transpose8x8(pack_bf16(fmaxf(rest.x, least.x), fmaxf(rest.y, least.y)));
        if (k & 1)
          pl[k >> 1].y = lo;
        else
          pl[k >> 1].x = lo;
      }
      p = transpose8x8(p);
      if (k & 1)
        pb[k >> 1].y = p;
      else
        pb[k >> 1].x = p;
    }
    // O^T += V^T P^T. Slots past the sequence's end may hold anything: their
    // values are zeroed in registers, since 0 * NaN would reach O.
#pragma unroll
    for (int u = 0; u < kUnit; ++u) {
      const uint32_t vb = stage + u * 2 * Cfg::kPlane + Cfg::kPlane;
      const int valid = keys - key0 - u * kPage;
      uint32_t mask[2] = {0xffffffffu, 0xffffffffu};
      if (valid < kPage) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          mask[h] = (half_key(h, 2 * tq) < valid ? 0x0000ffffu : 0u) |
                    (half_key(h, 2 * tq + 1) < valid ? 0xffff0000u : 0u);
      }
#pragma unroll
      for (int c = 0; c < (CODES ? 4 : 8); ++c) {
        uint32_t r[4];  // halves 0 and 1 of one chunk, then of the next
        ldsm_x4_t(vb + (CODES ? 0 : (c >> 2) * 2048) + off[c & 3], r);
        if (valid < kPage) {
          r[0] &= mask[0];
          r[1] &= mask[1];
          r[2] &= mask[0];
          r[3] &= mask[1];
        }
        if constexpr (CODES) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            // bytes (k0 d0, k0 d1, k1 d0, k1 d1) -> even dims (k0, k1), odd dims (k0, k1)
            uint4 A;
            widen4(__byte_perm(r[2 * h], 0u, 0x3120), A.x, A.y);
            widen4(__byte_perm(r[2 * h + 1], 0u, 0x3120), A.z, A.w);
            mma16816<true>(o[2 * c + h], A, pb[u]);
          }
        } else {
          const uint4 A = make_uint4(r[0], r[2], r[1], r[3]);
          mma16816<false>(o[c], A, pb[u]);
          mma16816<false>(o[c], A, pl[u]);
        }
      }
    }
    __syncwarp();  // every lane has read the stage
    if (issued < count) produce();
    if (cc.j == cc.n - 1 || i == count - 1) close_item();
    if (i < count - 1) next_unit<kUnit>(a, cc, lane);
  }

  if (!ok) {
    // Gave up: no copy, and no arrival that follows one, may land after the CTA's end.
    asm volatile("cp.async.wait_all;" ::: "memory");
    for (int k = max(0, issued - kStages); k < issued; ++k) {
      if (limit_clk < 0 && lane == 0) mbar_arrive(&bars[k % kStages]);
      const long long t0 = clock64();
      while (!mbar_try_wait(smem_u32(&bars[k % kStages]), static_cast<uint32_t>((k / kStages) & 1)) &&
             clock64() - t0 <= kWaitLimitCycles) {
      }
    }
    if (lane == 0) raise_device_error(a.c.err, QUAIL_ERR_DEVICE_TIMEOUT, 4000);
  }
}

// ------------------------------------------------------------------ join
// A row's parts, in this order: the prefix by key range (tiles), the prefix in
// pieces (streamed), the own keys in pieces (streamed) or by key range (tiles).
// Bound by latency: dependent reads (lengths, plan, parts), and the fetching of
// its instructions after hundreds of megabytes of keys have passed through L2.
// So it is short: lane i finds part i and reads its statistics, all at once, and
// one small loop adds the parts up. 8,192 rows of five parts: 10 us (12.4 with four
// rows to a warp, one after the other).
__device__ __forceinline__ float pow2_or_0(float x, float ref) {  // 2^(x - ref); 0 where nothing was seen
  return x == -INFINITY ? 0.f : exp2f(x - ref);
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int x = 1; x < 32; x <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, x));
  return v;
}

// The sum of up to 32 parts, one per lane (o: its 128 values; m_l = -inf: none):
// on return acc holds dims 4 lane .. 4 lane + 3, st the whole's statistics. The
// values of the first parts are read along with the statistics.
__device__ __forceinline__ float4 add_parts(const float* o, const PartStat* from, PartStat& st, int count, int lane) {
  auto value = [&](int i) {
    const float* p = reinterpret_cast<const float*>(
        __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(o), i));
    return *reinterpret_cast<const float4*>(p + 4 * lane);
  };
  st = lane < count ? *from : PartStat{-INFINITY, -INFINITY, 0.f, 0.f};
  constexpr int kFirst = 6;
  float4 v[kFirst];
#pragma unroll
  for (int i = 0; i < kFirst; ++i) v[i] = value(min(i, count - 1));
  const float ml = warp_max(st.m_l), mo = warp_max(st.m_o);
  const float f = pow2_or_0(st.m_o, mo);  // 0 in lanes past the last part
  float l = st.l != st.l ? st.l : st.l * pow2_or_0(st.m_l, ml);  // a NaN sum stays one, whatever its maximum
#pragma unroll
  for (int x = 1; x < 32; x <<= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](const float4& x, float w) {
    acc.x = fmaf(x.x, w, acc.x);
    acc.y = fmaf(x.y, w, acc.y);
    acc.z = fmaf(x.z, w, acc.z);
    acc.w = fmaf(x.w, w, acc.w);
  };
#pragma unroll
  for (int i = 0; i < kFirst; ++i) {
    const float w = __shfl_sync(0xffffffffu, f, i);
    if (i < count) add(v[i], w);
  }
#pragma unroll 4
  for (int i = kFirst; i < count; ++i) add(value(i), __shfl_sync(0xffffffffu, f, i));
  st = PartStat{mo, ml, l, 0.f};
  return acc;
}

// (st, acc) += (ps, v), two sums with their own maxima.
__device__ __forceinline__ void add_to(PartStat& st, float4& acc, const PartStat& ps, const float4& v) {
  const float ml = fmaxf(st.m_l, ps.m_l), mo = fmaxf(st.m_o, ps.m_o);
  const float f0 = pow2_or_0(st.m_o, mo), f1 = pow2_or_0(ps.m_o, mo);
  acc = make_float4(acc.x * f0 + v.x * f1, acc.y * f0 + v.y * f1, acc.z * f0 + v.z * f1, acc.w * f0 + v.w * f1);
  st.l = (st.l != st.l ? st.l : st.l * pow2_or_0(st.m_l, ml)) + (ps.l != ps.l ? ps.l : ps.l * pow2_or_0(ps.m_l, ml));
  st.m_l = ml;
  st.m_o = mo;
}

struct Parts {
  int prefix_dense, prefix_n, own_n, own_dense;
  uint32_t prefix_w, own_w;  // worker of the first piece
  int prefix_r, own_r;       // row within the items' tiles
};

// first and number of the workers of units [u, u + n)
__device__ __forceinline__ void pieces(long long u, int n, long long chunk, uint32_t* first, int* count) {
  if (u + n <= 0x7fffffffLL && chunk <= 0x7fffffffLL) {  // 32-bit division
    const uint32_t c = static_cast<uint32_t>(chunk), lo = static_cast<uint32_t>(u) / c;
    *first = lo;
    *count = static_cast<int>((static_cast<uint32_t>(u) + n - 1) / c - lo) + 1;
  } else {
    *first = static_cast<uint32_t>(u / chunk);
    *count = static_cast<int>((u + n - 1) / chunk - u / chunk) + 1;
  }
}

// The sequence whose queries row t is among, or -1, for all threads of the block. With
// many sequences every thread first asks for a run of them; only where no run has the
// row, or offsets that do not ascend hide it, are all looked at (sequences of 2 queries,
// 32 heads, all looked at / runs first: 1,024 43.5 / 45.4 us for the join, 4,096 of 4
// queries 353 / 307, 16,384 1,934 / 827, 65,535 25,142 / 3,426). A range that is none
// (query_range) has no row: it would take those of others.
template <int THREADS>
__device__ __forceinline__ int sequence_of(const SharedAttnArgs& a, int t, int* found) {
  const int n = a.c.num_seqs, per = (n + THREADS - 1) / THREADS;
  auto look = [&](int first, int end, int step) {  // step sequences at a time, the last that has the row
    if (threadIdx.x == 0) *found = -1;
    __syncthreads();
    for (int i = first + threadIdx.x * step; i < end; i += THREADS * step) {
      const int lo = a.q_offsets[i], hi = a.q_offsets[min(i + step, end)];
      if (lo <= t && t < hi && lo >= 0 && hi <= a.total_q && (step > 1 || hi - lo <= a.max_q)) *found = i;
    }
    __syncthreads();
    return *found;
  };
  if (per > 8) {
    const int run = look(0, n, per);
    __syncthreads();  // all have read it
    const int b = run < 0 ? -1 : look(run, min(run + per, n), 1);
    if (b >= 0) return b;
    __syncthreads();
  }
  return look(0, n, 1);
}

// PER_ROW: the block's WARPS warps share row blockIdx.x = token * hq + head, else
// each has a row, heads 8 blockIdx.y .. of token blockIdx.x.
template <bool PER_ROW, int WARPS>
__global__ void __launch_bounds__(32 * WARPS) attention_join_kernel(SharedAttnArgs a) {
  grid_dependency_wait();
  __shared__ float so[PER_ROW ? WARPS : 1][128];
  __shared__ PartStat ss[PER_ROW ? WARPS : 1];
  __shared__ int s_b;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.hq / a.c.hkv;
  const int t = PER_ROW ? blockIdx.x / a.hq : blockIdx.x;
  int b = t;
  if (a.q_offsets != nullptr) {
    b = sequence_of<32 * WARPS>(a, t, &s_b);
    if (b < 0) return;  // of no sequence: left as it was
  }
  const QueryRange qr = query_range(a, b);
  if (!qr.ok) return;
  const int unit = stream_unit_pages(a.c.codes);
  long long chunk = 1, base = 0;
  int n = 0, tiles = 0;
  if (a.streamed) {
    chunk = a.plan[1];
    base = a.plan[2 + b];
    n = qr.len > 0 ? (own_pages(a, b) + unit - 1) / unit : 0;
    tiles = own_items(a, b) / a.c.hkv;
  }
  const int pu = (a.prefix_len / kPage + unit - 1) / unit;
  for (int h = PER_ROW ? blockIdx.x % a.hq : blockIdx.y * WARPS + warp; h < a.hq; h += a.hq) {
    const int g = h / G;
    const size_t row = static_cast<size_t>(t) * a.hq + h;
    Parts p{};
    if (qr.len > 0) {
      const int r = (t - qr.lo) * G + h % G;
      p.prefix_dense = a.prefix_splits;
      if (a.streamed) {
        if (a.prefix_row_tiles > 0) {
          const int flat = t * G + h % G;
          pieces((static_cast<long long>(flat / kItemRows) * a.c.hkv + g) * pu, pu, chunk, &p.prefix_w, &p.prefix_n);
          p.prefix_r = flat % kItemRows;
        }
        if (n > 0) {
          pieces(base + (static_cast<long long>(g) * tiles + r / kItemRows) * n, n, chunk, &p.own_w, &p.own_n);
          p.own_r = r % kItemRows;
        }
        if (a.prefix_len == 0 && p.own_n == 1) continue;  // written by its only worker
      } else {
        const int keys = tile_key_end(a, qr, r) - a.seq_begin;
        p.own_dense = keys > 0 ? (keys + a.seq_split - 1) / a.seq_split : 0;
      }
    }
    const int parts = p.prefix_dense + p.prefix_n + p.own_n + p.own_dense;
    // this warp's parts, 32 at a time
    constexpr int kStep = PER_ROW ? WARPS : 1;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    PartStat st{-INFINITY, -INFINITY, 0.f, 0.f};
    const int mine = PER_ROW ? (parts - warp + WARPS - 1) / WARPS : parts;
    for (int i0 = 0; i0 < mine; i0 += 32) {
      const float* o = nullptr;
      const PartStat* from = nullptr;
      const int i = i0 + lane;
      if (i < mine) {
        int k = i * kStep + (PER_ROW ? warp : 0);
        size_t at = row;
        const float* po = a.dense_o;
        const PartStat* pst = a.dense_st;
        const int streamed = p.prefix_n + p.own_n;
        if (k < p.prefix_dense || k >= p.prefix_dense + streamed) {
          const int s = k < p.prefix_dense ? k : a.prefix_splits + k - p.prefix_dense - streamed;
          at += static_cast<size_t>(s) * a.total_q * a.hq;
        } else {
          k -= p.prefix_dense;
          const bool pre = k < p.prefix_n;
          const int piece = pre ? k : k - p.prefix_n;
          po = pre ? a.prefix_o : a.own_o;
          pst = pre ? a.prefix_st : a.own_st;
          if (piece > 0) {
            at = (static_cast<size_t>(pre ? p.prefix_w : p.own_w) + piece) * kItemRows + (pre ? p.prefix_r : p.own_r);
            po = a.cont_o;
            pst = a.cont_st;
          }
        }
        o = po + at * 128;
        from = pst + at;
      }
      PartStat ps;
      const float4 v = add_parts(o, from, ps, min(32, mine - i0), lane);
      add_to(st, acc, ps, v);
    }
    if constexpr (PER_ROW) {
      *reinterpret_cast<float4*>(&so[warp][4 * lane]) = acc;
      if (lane == 0) ss[warp] = st;
      __syncthreads();
      if (warp != 0) return;
      acc = add_parts(so[lane % WARPS], ss + lane % WARPS, st, WARPS, lane);
    }
    // no key at all: 0 and -inf. A NaN sum makes the row NaN, as the formula has it.
    const bool none = qr.len == 0;
    const float f = none ? 0.f : (st.l != st.l ? st.l : exp2f(st.m_o - st.m_l) / st.l);
    *reinterpret_cast<uint2*>(a.out + row * 128 + 4 * lane) =
        make_uint2(pack_bf16(acc.x * f, acc.y * f), pack_bf16(acc.z * f, acc.w * f));
    if (lane == 0 && a.lse != nullptr) a.lse[row] = none ? -INFINITY : (st.m_l + log2f(st.l)) * 0.6931471805599453f;
  }
}

}  // namespace

namespace {

template <bool CODES>
cudaError_t launch_stream(const SharedAttnArgs& a, int num_sms, cudaStream_t st) {
  auto kern = attention_stream_kernel<CODES>;
  constexpr size_t smem = StreamCfg<CODES>::kSmem;
  static std::atomic<bool> configured[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    configured[dev].store(true, std::memory_order_release);
  }
  count_launch();
  return launch_pdl(kern, dim3(num_sms), dim3(StreamCfg<CODES>::kThreads), smem, st, a);
}

}  // namespace

cudaError_t launch_attention_stream(const SharedAttnArgs& a, int num_sms, cudaStream_t st) {
  return a.c.codes ? launch_stream<true>(a, num_sms, st) : launch_stream<false>(a, num_sms, st);
}

cudaError_t launch_attention_join(const SharedAttnArgs& a, int num_sms, cudaStream_t st) {
  const long long rows = static_cast<long long>(a.total_q) * a.hq;
  count_launch();
  // Few rows have many parts (a streamed row up to all workers over the KV heads) and
  // leave SMs idle. Warps a row 16 / 4 / 1, us: 32 rows 13 / 23 / 46, 512 rows
  // 20 / 15 / 16, 1,024 rows 18 / 6.6 / 7.1, 2,048 rows 33 / 10 / 7.7, 8,192 rows
  // 103 / 30 / 10.
  if (rows <= num_sms)
    return launch_pdl(attention_join_kernel<true, 16>, dim3(static_cast<unsigned>(rows)), dim3(512), 0, st, a);
  if (rows <= 8LL * num_sms)
    return launch_pdl(attention_join_kernel<true, 4>, dim3(static_cast<unsigned>(rows)), dim3(128), 0, st, a);
  return launch_pdl(attention_join_kernel<false, 8>, dim3(a.total_q, (a.hq + 7) / 8), dim3(256), 0, st, a);
}

// Test hook: this translation unit's copy of the pipeline wait limit.
cudaError_t set_pipeline_wait_limit_cache_attention(long long cycles) {
  return cudaMemcpyToSymbol(g_pipeline_wait_limit, &cycles, sizeof(cycles));
}

}  // namespace quail
