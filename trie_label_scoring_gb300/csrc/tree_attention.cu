// Attention for trees of drafted tokens over the paged document cache: node i of a
// sequence's n sees the keys [0, len - n) and, of the last n, those that its mask row has
// bits for:  o = softmax(scale q K^T) V,  lse = log sum exp(scale q K^T).
//
// Dozens of query rows per KV head (nodes times heads of a group), keys by the thousand:
// the keys and values are to be read once, and the few rows should cost little beside them.
// So the keys take the 128 rows of the tensor core's tile and the queries its columns, N =
// 16 to 128 of them, on tcgen05:
//   S^T = K Q^T    M 128 keys, N query rows, K 128 dims
//   O^T += V^T P^T M 128 dims, N query rows, K 128 keys
// (an instruction takes 46 clocks up to 32 columns, 49 for 64, 65 for 128,
// whichever way its operands lie in shared memory). K and V pages go from memory to the
// products as they lie: V^T is V read along its rows. A thread of the softmax has one key
// and 32 scores: a key's own factors are scalars of its thread, and no row waits for a
// shuffle. The maximum of a query row would need one, over all 128 keys; so rows keep a
// reference that moves only when some score passes it by a margin (2^8, codes 2^4), and the
// sums of the weights stay in the threads until the end. Whether one does is a vote of the
// four warps that runs while they take the weights; the block that moves a reference (the
// first of a piece, then one in thirty with codes) takes them again. P^T is laid into shared
// memory key by key.
//
// Over an e4m3 cache the codes are operands as they are (kind::f8f6f4): no widening. A query
// element, 8 significant bits, is an e4m3 and an e5m2 term exactly (down to 2^-17 of the
// row's largest; below, off by up to 2^-21 of it); a weight, times its value row's power of
// two, is cut into three e5m2 terms, 9 bits. e5m2 because its exponents reach from 2^-16 to
// 2^15: weights are taken times 2^11, at most 2^15, and lost below 2^-28 of the largest
// weight times the largest power. The terms come out of an fp16's upper bytes: converting
// fp32 to e5m2 three times took 238 us where this takes 202 (32 sequences of 24 nodes).
// Over a bf16 cache a weight is two bf16 terms up to 32 columns (o's error is that of its
// own rounding, 0.0017 relative) and one beyond (0.0023; with two, and two barriers a block
// more, the first case below took 65 us).
// Up to 64 columns a weight's terms are columns of one product, with sums of their own.
//
// Work: an item is a (sequence, KV head, row tile), its blocks 128 keys each. Where no
// sequence is long the CTAs take whole items in turn, and nothing is left to join. Else the
// blocks of all items, with three units ahead of each for what an item costs to begin and
// end, are one list that is cut into equal runs, one per CTA, whatever the lengths are, and
// the pieces of an item that several CTAs share are joined by a second kernel, which comes up
// beside the last of these CTAs.
//
// What bounds it. 64 sequences of 1 to 12 nodes, 128 to 2,048 keys (32 heads on 8): 59 us,
// 4.9 TB/s; a block takes 2,200 clocks where reading its 64 KB takes 2,900 at full rate, so
// memory is what counts, and a piece another 5,000 to begin and end, in part hidden by the
// pages that come in meanwhile. 16 sequences of 40 to 100 nodes, 1,024 to 4,096 keys: 94 us,
// three or four tiles of 96 columns; 32 of 24 nodes over 7,000 to 8,192 codes: 167 us. There a
// block takes 2,600 and 3,000 clocks, the softmax: three warps a scheduler issue 40 and 52%
// of the time, each an instruction in 6 to 8 clocks (latency of dependent instructions); with
// codes 520 instructions of a warp and block, 28% of them the terms, and the ALU pipe 40% busy.
//
// Roles: warp 0 and 3 load K and V pages (TMA, a page a lane), warp 1 issues the products,
// warp 2 walks the work list, publishes its pieces and loads bf16 queries, warps 4.. are
// the softmax, a warpgroup per 32 columns (a thread per key of a block, per dim of O). Its
// barriers are mbarriers like all others here, so that a wait that gives up ends them all.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "cache_attn.cuh"
#include "launch.cuh"
#include "quail_internal.h"
#include "sm103.cuh"
#include "tree.h"

namespace quail {

namespace {

constexpr int kBlk = 128;  // keys of a block
constexpr int kBlkPages = kBlk / kPage;
constexpr int kPieces = 4;  // published ahead
constexpr float kNone = 3e38f;  // minus the reference of a row that has seen no key

template <int N, bool CODES>
struct Cfg {
  static constexpr int kCols = N < 32 ? N : 32;  // columns of a softmax warpgroup
  static constexpr int kWgs = N / kCols;
  static constexpr int kThreads = 128 + 128 * kWgs;
  static constexpr int kTerms = CODES ? 3 : N > 32 ? 1 : 2;  // of a weight
  static constexpr uint32_t kRow = CODES ? 128 : 256;  // bytes of a key
  static constexpr uint32_t kSlot = kBlk * kRow;
  static constexpr int kDepth = !CODES ? 2 : N == 96 ? 3 : 4;   // blocks of K, and of V, in flight or at work
  static constexpr uint32_t kHalf = CODES ? 0 : kBlk * 128;  // bf16: 64 dims of a block's rows
  static constexpr uint32_t kQ = N * 256;        // two halves of bf16, or two terms of codes
  // P: rows of 128 bytes by key, in blocks of 128 keys; the terms side by side in a block's
  // rows where they fit
  static constexpr int kColBytes = CODES ? 1 : 2;
  static constexpr int kTermBytes = N == 96 ? (CODES ? 128 : 256) : N * kColBytes;
  static constexpr int kPBlock = kBlk * 128;
  static constexpr int kPBlocks = (kTermBytes * kTerms + 127) / 128;
  static constexpr uint32_t kP = kPBlocks * kPBlock;
  static constexpr int kPBufs = N == 128 ? 1 : 2;
  static constexpr uint32_t kOffV = kDepth * kSlot;
  static constexpr uint32_t kOffQ = kOffV + kDepth * kSlot;
  static constexpr uint32_t kOffP = kOffQ + kQ;
  static constexpr uint32_t kOffStats = kOffP + kPBufs * kP;
  // The terms of a weight as columns of one product, with sums of their own, where that makes
  // it no wider than an instruction (which takes at least 46 clocks, as for 32 columns); else
  // one after the other into the same sums.
  static constexpr bool kWide = N <= 64;
  static constexpr int kOCols = kWide ? kTerms * N : N;
  static constexpr int kTmemUsed = 2 * N + kOCols;  // two S, one O
  static constexpr int kTmem = kTmemUsed <= 64 ? 64 : kTmemUsed <= 128 ? 128 : kTmemUsed <= 256 ? 256 : 512;
  static constexpr int kMargin = CODES ? 4 : 8;  // a score may pass the reference by, base 2
  static constexpr int kLift = 11;               // of codes' weights
};

struct Piece {
  int b, g;
  int lo, n, len;  // the tree's first row, its nodes, the sequence's keys
  int tok0;        // first node of the row tile
  int blk0, blks;  // blocks of keys; blks 0: no key at all, < 0: no more pieces
  int slot;        // where its rows go: -1 the result itself, 0 and 1 this CTA's parts
};

template <int N, bool CODES>
struct Shared {
  float neg_ref[Cfg<N, CODES>::kWgs][4][Cfg<N, CODES>::kCols];  // minus the reference maxima, every warp's own copy
  float row_factor[N]; // codes: score factor times the query row's power of two
  // maxima or sums of a warp's keys, in turn by the warpgroup's barriers: what was written
  // before one is read before the next, and written over behind that
  float part[Cfg<N, CODES>::kWgs][2][4][Cfg<N, CODES>::kCols];
  int part_e[Cfg<N, CODES>::kWgs][2][4];
  struct {
    int row;  // of the result, -1: none
    float factor;
  } last[Cfg<N, CODES>::kWgs][4][Cfg<N, CODES>::kCols];
  int moved[Cfg<N, CODES>::kWgs][2];  // block, plus one, for which a warp asks to move the reference
  Piece piece[kPieces];
  uint64_t piece_full[kPieces], piece_empty[kPieces];
  uint64_t k_full[Cfg<N, CODES>::kDepth], k_empty[Cfg<N, CODES>::kDepth];
  uint64_t v_full[Cfg<N, CODES>::kDepth], v_empty[Cfg<N, CODES>::kDepth];
  uint64_t q_full, q_empty, s_full[2], p_full[2], p_empty[2], drain;
  uint64_t vote[Cfg<N, CODES>::kWgs][2], wg_sync[Cfg<N, CODES>::kWgs];
  uint32_t tmem;
  int abort_flag;
};
template <int N, bool CODES>
constexpr size_t tree_smem() {
  constexpr size_t n = 1024 + Cfg<N, CODES>::kOffStats + sizeof(Shared<N, CODES>);
  static_assert(n <= 227 * 1024, "shared memory");
  return n;
}

// ------------------------------------------------------------------ small parts
struct Seq {
  int lo, n, len;
  bool ok;
};
__device__ __forceinline__ Seq seq_of(const TreeAttnArgs& a, int b) {
  Seq s;
  s.lo = a.q_offsets[b];
  s.n = a.q_offsets[b + 1] - s.lo;
  s.len = a.seq_len[b];
  s.ok = s.lo >= 0 && s.n >= 0 && s.n <= a.max_q && s.lo <= a.total_q - s.n && s.len >= 0 && s.len <= a.max_seq_len &&
         (s.len == 0 || s.len >= s.n);
  return s;
}
__device__ __forceinline__ int blocks_of(int len) { return (len + kBlk - 1) / kBlk; }
// Units of a sequence in the work list, and its (head, row tile) items: an item is kBegin
// units, what it costs to begin and end it, and then its blocks.
constexpr int kBegin = 3;
__device__ __forceinline__ long long units_of(const TreeAttnArgs& a, int b, int* items) {
  const Seq s = b < a.c.num_seqs ? seq_of(a, b) : Seq{0, 0, 0, false};
  *items = s.ok ? (s.n + a.tile_tokens - 1) / a.tile_tokens * a.c.hkv : 0;
  return s.ok && s.len > 0 ? static_cast<long long>(blocks_of(s.len) + kBegin) * *items : 0;
}

__device__ __forceinline__ void umma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Instruction descriptors: fp32 D; kind::f16 with bf16, or kind::f8f6f4 with e4m3 A and B of
// either type. Bits 15 and 16: A, B along their M, N.
constexpr uint32_t kAlongM = 1u << 15, kAlongN = 1u << 16;
__host__ __device__ constexpr uint32_t idesc_f8(int N, bool b_e5m2) {
  return (1u << 4) | (b_e5m2 ? 1u << 10 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) | (8u << 24);
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* tm, uint64_t* bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// C columns of this thread's TMEM lane (16 or 32), waited for.
template <int C>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, float (&v)[C]) {
  uint32_t r[C];
  if constexpr (C == 32) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
  } else {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
  }
#pragma unroll
  for (int i = 0; i < C; ++i) v[i] = __uint_as_float(r[i]);
}
template <int C>
__device__ __forceinline__ void tmem_st_cols(uint32_t taddr, const float (&v)[C]) {
  if constexpr (C == 32) {
    tmem_st_32cols(taddr, v);
  } else {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};\n\t"
        "tcgen05.wait::st.sync.aligned;" ::"r"(taddr),
        "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3])),
        "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])), "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7])),
        "r"(__float_as_uint(v[8])), "r"(__float_as_uint(v[9])), "r"(__float_as_uint(v[10])),
        "r"(__float_as_uint(v[11])), "r"(__float_as_uint(v[12])), "r"(__float_as_uint(v[13])),
        "r"(__float_as_uint(v[14])), "r"(__float_as_uint(v[15]))
        : "memory");
  }
}

// `width` bits from bit `lo` on, as far as there are 32.
__device__ __forceinline__ uint32_t bits_from(int lo, int width) {
  uint32_t r;
  asm("bmsk.clamp.b32 %0, %1, %2;" : "=r"(r) : "r"(lo), "r"(width));
  return r;
}

// Column i of v over the warp's lanes, to lane i (mod C): each step halves the columns a
// lane keeps and doubles the lanes that they stand for.
template <int C, class Op>
__device__ __forceinline__ float over_lanes(float (&v)[C], int lane, Op op) {
  if constexpr (C == 16) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = op(v[i], __shfl_xor_sync(0xffffffffu, v[i], 16));
  }
#pragma unroll
  for (int d = C / 2; d > 0; d >>= 1) {
    const bool upper = (lane & d) != 0;
#pragma unroll
    for (int i = 0; i < d; ++i) {
      const float keep = upper ? v[i + d] : v[i], give = upper ? v[i] : v[i + d];
      v[i] = op(keep, __shfl_xor_sync(0xffffffffu, give, d));
    }
  }
  return v[0];
}

__device__ __forceinline__ uint32_t e5m2x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t v) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(v)));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// Blocks up to the last one that some node of the row tile sees, one at least: in a tree
// larger than a block, ancestors come first, so the tiles of its early nodes end early. By a
// whole warp.
__device__ __forceinline__ int blocks_seen(const TreeAttnArgs& a, const Seq& s, int tok0, int lane) {
  if (s.n <= kBlk) return blocks_of(s.len);
  const int used = (s.n + 31) / 32, words = min(a.tile_tokens, s.n - tok0) * used;
  const uint32_t* rows = a.mask + static_cast<size_t>(s.lo + tok0) * a.words;
  int top = -1;
#pragma unroll 4
  for (int i = lane; i < words; i += 32) {
    const int w = i % used;
    uint32_t m = rows[i / used * a.words + w];
    if (w == used - 1 && s.n % 32 != 0) m &= (1u << (s.n % 32)) - 1;
    if (m != 0) top = max(top, w);
  }
  top = __reduce_max_sync(0xffffffffu, top);
  return max(1, blocks_of(min(s.len, s.len - s.n + 32 * (top + 1))));
}

// 2^e for any e, 0 and infinity past the ends.
__device__ __forceinline__ float pow2_int(int e) {
  return e < -126 ? 0.f : e > 127 ? INFINITY : __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// ------------------------------------------------------------------ the kernel
template <int N, bool CODES>
__global__ void __launch_bounds__(Cfg<N, CODES>::kThreads, 1)
    tree_attention_kernel(TreeAttnArgs a, const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                          const __grid_constant__ CUtensorMap tmQ) {
  using C = Cfg<N, CODES>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = smem_raw + (-smem_u32(smem_raw) & 1023u);
  auto& sh = *reinterpret_cast<Shared<N, CODES>*>(base + C::kOffStats);
  volatile int* abort_flag = &sh.abort_flag;
  const long long limit_clk = pipeline_wait_limit();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.hq / a.c.hkv;
  grid_dependency_wait();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kPieces; ++s) {
      mbar_init(&sh.piece_full[s], 1);
      mbar_init(&sh.piece_empty[s], 3 + 4 * C::kWgs);  // the loaders, the issuer, the softmax warps
    }
    for (int s = 0; s < C::kDepth; ++s) {
      mbar_init(&sh.k_full[s], 1);
      mbar_init(&sh.k_empty[s], 1);
      mbar_init(&sh.v_full[s], 1);
      mbar_init(&sh.v_empty[s], 1);
    }
    mbar_init(&sh.q_full, CODES ? 4 * C::kWgs : 1);
    mbar_init(&sh.q_empty, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sh.s_full[s], 1 + (limit_clk < 0));
      mbar_init(&sh.p_full[s], 4 * C::kWgs);
      mbar_init(&sh.p_empty[s], 1);
    }
    mbar_init(&sh.drain, 1);
    for (int g = 0; g < C::kWgs; ++g) {
      mbar_init(&sh.vote[g][0], 4);
      mbar_init(&sh.vote[g][1], 4);
      mbar_init(&sh.wg_sync[g], 4);
      sh.moved[g][0] = sh.moved[g][1] = 0;
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  // query columns without a row: zeros, so that their scores are finite
  for (uint32_t i = threadIdx.x; i < C::kQ / 16; i += C::kThreads)
    reinterpret_cast<uint4*>(base + C::kOffQ)[i] = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();

  // ---- the plan: thread i counts the blocks of its own run of sequences
  long long chunk = 0, u0 = 0, count = 0;  // blocks of a run; this CTA's
  int b_at = 0, x_at = 0, j_at = 0;
  if (!a.direct) {
    long long* scan = reinterpret_cast<long long*>(base + C::kOffP);  // kThreads + 1 of them
    const int B = a.c.num_seqs, per = (B + C::kThreads - 1) / C::kThreads;
    const int b0 = min(B, static_cast<int>(threadIdx.x) * per), b1 = min(B, b0 + per);
    long long mine = 0;
    for (int b = b0; b < b1; ++b) {
      if (blockIdx.x == 0 && !seq_of(a, b).ok) raise_device_error(a.c.err, QUAIL_ERR_DEVICE_BOUNDS, b);
      int items;
      mine += units_of(a, b, &items);
    }
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
    const long long units = scan[C::kThreads];
    // two at least: a part per block is more to join than it saves (5,205 keys of one head 15.1 us, 13.7)
    chunk = max(2LL, (units + gridDim.x - 1) / gridDim.x);
    u0 = blockIdx.x * chunk;
    count = max(0LL, min(units, u0 + chunk) - u0);
    if (warp == 2 && count > 0) {  // where the run begins
      int lo = 0, hi = C::kThreads;  // scan[lo] <= u0 < scan[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (scan[mid] <= u0)
          lo = mid;
        else
          hi = mid;
      }
      long long at = scan[lo];
      for (int b = lo * per;; ++b) {
        int items;
        const long long n = units_of(a, b, &items);
        if (at + n > u0 || b >= B) {
          const int per_item = (b < B ? blocks_of(a.seq_len[b]) : 0) + kBegin;
          b_at = b;
          x_at = static_cast<int>((u0 - at) / per_item);
          j_at = static_cast<int>((u0 - at) % per_item);
          break;
        }
        at += n;
      }
    }
  }
  __syncthreads();
  // the join, which takes no tensor memory, may come up beside this kernel's CTAs; it waits
  // for their end
  if (!a.direct) grid_launch_dependents();

  // ---- a role's way along the pieces
  int piece_no = 0;
  auto piece_there = [&]() {
    return __all_sync(0xffffffffu, wait_bar(&sh.piece_full[piece_no % kPieces], static_cast<uint32_t>((piece_no / kPieces) & 1), abort_flag, limit_clk)) != 0;
  };
  auto take_piece = [&](Piece& p) {
    if (!piece_there()) return false;
    p = sh.piece[piece_no % kPieces];
    return true;
  };
  auto done_piece = [&]() {  // one arrival a warp
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.piece_empty[piece_no % kPieces]);
    ++piece_no;
  };
  // the n-th use of one of `of` stages of a ring: waits for its phase
  auto wait_use = [&](uint64_t* bars, int of, int n) {
    return wait_bar(&bars[n % of], static_cast<uint32_t>((n / of) & 1), abort_flag, limit_clk);
  };
  // a wait that no abort cuts short: copies and products in flight
  auto wait_landed = [&](uint64_t* bar, uint32_t parity) {
    const long long t0 = clock64();
    while (!mbar_try_wait(smem_u32(bar), parity)) {
      if (clock64() - t0 > kWaitLimitCycles) {
        *abort_flag = 1;
        break;
      }
    }
  };

  if (warp == 2) {
    // ------------------------------------------------ the work list
    int published = 0, q_loads = 0;
    bool ok = true;
    auto publish = [&](const Piece& p) {
      const int s = published % kPieces;
      if (published >= kPieces)
        ok = __all_sync(0xffffffffu, wait_use(sh.piece_empty, kPieces, published - kPieces));
      if (!ok) return;
      if (lane == 0) {
        sh.piece[s] = p;
        mbar_arrive(&sh.piece_full[s]);
      }
      ++published;
      if (!CODES && p.blks > 0) {
        if (q_loads > 0) ok = __all_sync(0xffffffffu, wait_use(&sh.q_empty, 1, q_loads - 1));
        if (!ok) return;
        if (lane == 0) {
          mbar_arrive_expect_tx(&sh.q_full, 2 * 128 * G * a.tile_tokens);
          tma_load_3d(base + C::kOffQ, &tmQ, &sh.q_full, 0, p.g * G, p.lo + p.tok0);
          tma_load_3d(base + C::kOffQ + N * 128, &tmQ, &sh.q_full, 64, p.g * G, p.lo + p.tok0);
        }
        ++q_loads;
      }
      __syncwarp();
    };
    Piece p{};
    if (a.direct) {
      const int tiles = (a.max_q + a.tile_tokens - 1) / a.tile_tokens, per_seq = a.c.hkv * tiles;
      const long long items = static_cast<long long>(a.c.num_seqs) * per_seq;
      for (long long i = blockIdx.x; ok && i < items; i += gridDim.x) {
        p.b = static_cast<int>(i / per_seq);
        const int x = static_cast<int>(i % per_seq);
        const Seq s = seq_of(a, p.b);
        if (!s.ok) {
          if (x == 0 && lane == 0) raise_device_error(a.c.err, QUAIL_ERR_DEVICE_BOUNDS, p.b);
          continue;
        }
        p.g = x / tiles;
        p.tok0 = x % tiles * a.tile_tokens;
        if (p.tok0 >= s.n) continue;
        p.lo = s.lo;
        p.n = s.n;
        p.len = s.len;
        p.blk0 = 0;
        p.blks = s.len > 0 ? blocks_seen(a, s, p.tok0, lane) : 0;
        p.slot = -1;
        publish(p);
      }
    } else {
      long long left = count;
      SharedItem begun{0, 0, 0, 0};  // the item that this CTA begins and leaves
      for (int b = b_at, x = x_at, j = j_at; ok && left > 0; ++b, x = 0) {
        // the next sequence with keys and nodes, 32 looked at at a time
        for (; b < a.c.num_seqs; b += 32) {
          int n;
          const uint32_t some = __ballot_sync(0xffffffffu, units_of(a, b + lane, &n) > 0);
          if (some != 0) {
            b += __ffs(some) - 1;
            break;
          }
        }
        if (b >= a.c.num_seqs) break;
        const Seq s = seq_of(a, b);
        const int tiles = (s.n + a.tile_tokens - 1) / a.tile_tokens, blks = blocks_of(s.len);
        p.b = b;
        p.lo = s.lo;
        p.n = s.n;
        p.len = s.len;
        for (; ok && left > 0 && x < tiles * a.c.hkv; ++x, j = 0) {
          const int units = static_cast<int>(min(left, static_cast<long long>(blks + kBegin - j)));
          p.g = x / tiles;
          p.tok0 = x % tiles * a.tile_tokens;
          const int seen = blocks_seen(a, s, p.tok0, lane);  // what lies behind is nobody's
          p.blk0 = max(0, j - kBegin);
          p.blks = min(seen, max(0, j + units - kBegin)) - p.blk0;
          p.slot = p.blks == seen ? -1 : p.blk0 > 0 ? 1 : 0;
          if (p.blks > 0) publish(p);
          if (p.blks > 0 && p.slot == 0)
            begun = SharedItem{s.lo + p.tok0, min(a.tile_tokens, s.n - p.tok0), p.g,
                               1 + static_cast<int>((seen - p.blks + chunk - 1) / chunk)};
          left -= units;
        }
      }
      if (lane == 0) a.shared_items[blockIdx.x] = begun;
    }
    p.blks = -1;
    if (ok) publish(p);
    if (!CODES && q_loads > 0) wait_landed(&sh.q_full, static_cast<uint32_t>((q_loads - 1) & 1));
  } else if (warp == 0 || warp == 3) {
    // ------------------------------------------------ loaders (K: warp 0, V: warp 3)
    // Lane q takes page q of a block; the ids of the next block are read while this one
    // waits for its slot.
    const CUtensorMap* tm = warp == 0 ? &tmK : &tmV;
    uint64_t* full = warp == 0 ? sh.k_full : sh.v_full;
    uint64_t* empty = warp == 0 ? sh.k_empty : sh.v_empty;
    uint8_t* ring = base + (warp == 0 ? 0 : C::kOffV);
    if (lane == 0) tma_prefetch_desc(tm);
    int t = 0;  // blocks issued
    bool ok = true;
    Piece p;
    while (ok && take_piece(p)) {
      done_piece();
      if (p.blks < 0) break;
      const int* table = a.c.table + static_cast<size_t>(p.b) * a.c.max_pages;
      const int pages = (p.len + kPage - 1) / kPage;
      auto page_id = [&](int blk) {
        const int i = (p.blk0 + blk) * kBlkPages + lane;
        return blk < p.blks && lane < kBlkPages && i < pages ? table[i] : -1;
      };
      int next = page_id(0);
      for (int j = 0; j < p.blks; ++j, ++t) {
        int page = next;
        next = page_id(j + 1);
        const bool mine = lane < kBlkPages && (p.blk0 + j) * kBlkPages + lane < pages;
        if (mine && (page < 0 || page >= a.c.num_pages)) {
          raise_device_error(a.c.err, QUAIL_ERR_DEVICE_BOUNDS, p.b);
          page = -1;  // not copied: the slot's old contents are consumed, the rows are void
        }
        const uint32_t good = __popc(__ballot_sync(0xffffffffu, page >= 0));
        const int s = t % C::kDepth;
        if (t >= C::kDepth && !__all_sync(0xffffffffu, wait_use(empty, C::kDepth, t - C::kDepth))) {
          ok = false;
          break;
        }
        if (lane == 0) {
          if (good > 0)
            mbar_arrive_expect_tx(&full[s], good * kPage * C::kRow);
          else
            mbar_arrive(&full[s]);
        }
        __syncwarp();
        if (page >= 0) {
          const int y = (page * a.c.hkv + p.g) * kPage;
          uint8_t* dst = ring + s * C::kSlot + lane * 2048;
          tma_load_2d(dst, tm, &full[s], 0, y);
          if constexpr (!CODES) tma_load_2d(dst + C::kHalf, tm, &full[s], 64, y);
        }
      }
    }
    // no copy may still be landing when the CTA exits
    for (int i = max(0, t - C::kDepth); lane == 0 && i < t; ++i)
      wait_landed(&full[i % C::kDepth], static_cast<uint32_t>((i / C::kDepth) & 1));
  } else if (warp == 1) {
    // ------------------------------------------------ issuer of the products
    tmem_alloc(&sh.tmem, C::kTmem);
    tmem_relinquish();
    tc_fence_before();
    asm volatile("bar.sync 1, %0;" ::"n"(32 + 128 * C::kWgs) : "memory");
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    const uint64_t dk = smem_desc_sw128(smem_u32(base)), dq = smem_desc_sw128(smem_u32(base + C::kOffQ));
    const uint64_t dv = smem_desc_sw128_mn(smem_u32(base + C::kOffV), CODES ? 1024 : C::kHalf, 1024);
    const uint64_t dp = smem_desc_sw128_mn(smem_u32(base + C::kOffP), C::kPBlock, 1024);
    auto issue_s = [&](int t) {
      const uint64_t k = dk + ((t % C::kDepth * C::kSlot) >> 4);
      const uint32_t d = tmem + (t & 1) * N;
      if constexpr (CODES) {
#pragma unroll
        for (int term = 0; term < 2; ++term)
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)  // 32 dims an instruction
            umma_f8(d, k + ((ks * 32) >> 4), dq + ((term * N * 128 + ks * 32) >> 4), idesc_f8(N, term == 1), term + ks != 0);
      } else {
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)  // 16 dims
          umma_bf16(d, k + (((ks >> 2) * C::kHalf + (ks & 3) * 32) >> 4), dq + (((ks >> 2) * N * 128 + (ks & 3) * 32) >> 4),
                    umma_idesc_bf16_f32(128, N), ks != 0);
      }
    };
    auto issue_pv = [&](int t, bool first) {
      const uint64_t v = dv + ((t % C::kDepth * C::kSlot) >> 4), w = dp + ((t % C::kPBufs * C::kP) >> 4);
      const uint32_t d = tmem + 2 * N;
#pragma unroll
      for (int term = 0; term < (C::kWide ? 1 : C::kTerms); ++term) {
        constexpr int kKeys = CODES ? 32 : 16;  // an instruction's
        const int at = term * C::kTermBytes, off = at / 128 * C::kPBlock + at % 128;
#pragma unroll
        for (int kk = 0; kk < kBlk / kKeys; ++kk) {
          const uint64_t av = v + ((kk * kKeys * 128) >> 4), bp = w + ((off + kk * kKeys * 128) >> 4);
          const uint32_t acc = !first || term + kk != 0;
          if constexpr (CODES)
            umma_f8(d, av, bp, idesc_f8(C::kOCols, true) | kAlongM | kAlongN, acc);
          else
            umma_bf16(d, av, bp, umma_idesc_bf16_f32(128, C::kOCols) | kAlongM | kAlongN, acc);
        }
      }
    };
    int t = 0, q_uses = 0;  // blocks; pieces with queries
    bool ok = true;
    Piece p;
    while (ok && take_piece(p)) {
      done_piece();
      if (p.blks < 0) break;
      if (p.blks == 0) continue;
      if (lane == 0) {
        auto scores = [&](int j) {
          ok = wait_use(sh.k_full, C::kDepth, t + j);
          if (!ok) return;
          tc_fence_after();
          issue_s(t + j);
          umma_commit(&sh.s_full[(t + j) & 1]);
          umma_commit(&sh.k_empty[(t + j) % C::kDepth]);
          if (!CODES && j == p.blks - 1) umma_commit(&sh.q_empty);
        };
        ok = wait_use(&sh.q_full, 1, q_uses);
        if (ok) scores(0);
        for (int j = 0; ok && j < p.blks; ++j) {
          if (j + 1 < p.blks) scores(j + 1);
          ok = ok && wait_use(sh.v_full, C::kDepth, t + j) && wait_use(sh.p_full, C::kPBufs, t + j);
          if (!ok) break;
          tc_fence_after();
          issue_pv(t + j, j == 0);
          umma_commit(&sh.p_empty[(t + j) % C::kPBufs]);
          umma_commit(&sh.v_empty[(t + j) % C::kDepth]);
        }
      }
      ok = __shfl_sync(0xffffffffu, static_cast<int>(ok), 0) != 0;
      ++q_uses;
      t += p.blks;
    }
    // every product of this thread completes before tensor memory is released
    if (lane == 0) {
      umma_commit(&sh.drain);
      wait_landed(&sh.drain, 0);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------ softmax: thread <-> key of a block, dim of O
    constexpr int W = C::kCols;
    const int wg = (warp - 4) >> 2, quarter = warp & 3, row = quarter * 32 + lane, c0 = wg * W;
    tc_fence_before();
    asm volatile("bar.sync 1, %0;" ::"n"(32 + 128 * C::kWgs) : "memory");
    tc_fence_after();
    const uint32_t tmem = sh.tmem + (static_cast<uint32_t>(quarter * 32) << 16), o_at = tmem + 2 * N + c0;
    auto wait_warp = [&](uint64_t* bars, int of, int n) { return __all_sync(0xffffffffu, wait_use(bars, of, n)) != 0; };
    // The warpgroup's barrier; like every wait here it ends when another role has given up.
    int syncs = 0;
    auto sync_warpgroup = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.wg_sync[wg]);
      return wait_warp(&sh.wg_sync[wg], 1, syncs++);
    };
    float* neg_ref = sh.neg_ref[wg][quarter];
    int t = 0;
    while (piece_there()) {
      const Piece& p = sh.piece[piece_no % kPieces];  // until done_piece
      const int blks = p.blks;
      if (blks < 0) break;
      // the result's row of this lane's column (of the warpgroup's)
      const int c = lane % W, c_node = (c0 + c) / G;
      const bool c_there = c_node < a.tile_tokens && p.tok0 + c_node < p.n;
      const int c_row = c_there ? (p.lo + p.tok0 + c_node) * a.hq + p.g * G + (c0 + c) % G : -1;
      if (blks == 0) {  // no key: zeros
        for (int i = 0; i < W; ++i) {
          const int r = __shfl_sync(0xffffffffu, c_row, i);
          if (r >= 0) a.out[static_cast<size_t>(r) * 128 + row] = __float2bfloat16(0.f);
        }
        if (quarter == 0 && lane < W && c_there && a.lse != nullptr) a.lse[c_row] = -INFINITY;
        done_piece();
        continue;
      }
      if constexpr (CODES) {
        // the warpgroup's query rows as two terms, 128 / W threads a row
        constexpr int kTpr = 128 / W, kPer = 128 / kTpr;  // threads a row, elements a thread
        const int qc = c0 + row / kTpr, part = row % kTpr, node = qc / G;
        uint4 x[kPer / 8];
        const bool there = node < a.tile_tokens && p.tok0 + node < p.n;
        const uint4* src = reinterpret_cast<const uint4*>(
            a.q + (static_cast<size_t>(p.lo + p.tok0 + (there ? node : 0)) * a.hq + p.g * G + (there ? qc % G : 0)) * 128 + part * kPer);
#pragma unroll
        for (int i = 0; i < kPer / 8; ++i) x[i] = there ? src[i] : make_uint4(0u, 0u, 0u, 0u);
        float am = 0.f;
        bool odd = false;  // an infinity or a NaN
        const uint32_t* xw = reinterpret_cast<const uint32_t*>(x);
#pragma unroll
        for (int i = 0; i < kPer / 2; ++i) {
          const float2 v = unpack_bf16(xw[i]);
          odd = odd || !(fabsf(v.x) < INFINITY) || !(fabsf(v.y) < INFINITY);
          am = fmaxf(am, fmaxf(fabsf(v.x), fabsf(v.y)));
        }
        uint32_t odd_row = odd;
#pragma unroll
        for (int d = 1; d < kTpr; d <<= 1) {
          am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, d));
          odd_row |= __shfl_xor_sync(0xffffffffu, odd_row, d);
        }
        // times 2^(7 - e): the largest in [128, 256)
        const int e = am > 0.f && !odd_row ? min(127, max(-119, static_cast<int>(__float_as_uint(am) >> 23) - 127)) : 0;
        const float up = pow2_int(7 - e);
        uint8_t* q0 = base + C::kOffQ + qc * 128;
#pragma unroll
        for (int i = 0; i < kPer / 16; ++i) {
          uint32_t w0[4], w1[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t hi[2], lo[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float2 v = unpack_bf16(xw[8 * i + 2 * k + h]);
              v = make_float2(v.x * up, v.y * up);
              hi[h] = e4m3x2(v.x, v.y);
              const float2 back = from_e4m3x2(hi[h]);
              lo[h] = e5m2x2(v.x - back.x, v.y - back.y);
            }
            w0[k] = odd_row ? 0x7f7f7f7fu : hi[0] | hi[1] << 16;
            w1[k] = odd_row ? 0u : lo[0] | lo[1] << 16;
          }
          const int chunk = (part * kPer / 16 + i) ^ (qc & 7);
          *reinterpret_cast<uint4*>(q0 + (chunk << 4)) = make_uint4(w0[0], w0[1], w0[2], w0[3]);
          *reinterpret_cast<uint4*>(q0 + N * 128 + (chunk << 4)) = make_uint4(w1[0], w1[1], w1[2], w1[3]);
        }
        if (part == 0) sh.row_factor[qc] = fmaxf(a.scale_log2 * pow2_int(e - 7), 1.17549435e-38f);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.q_full);
        if (!sync_warpgroup()) break;
      }
      float2 l[W / 2];  // this key lane's sums
#pragma unroll
      for (int i = 0; i < W / 2; ++i) l[i] = make_float2(0.f, 0.f);
      int e_ref = 0;  // codes: the largest power of the values seen, biased
      // codes: this thread's key's powers, read a block ahead, its page's id two
      auto page_id = [&](int j) {
        const int key = (p.blk0 + j) * kBlk + row;
        return j < blks && key < p.len ? a.c.table[static_cast<size_t>(p.b) * a.c.max_pages + key / kPage] : -1;
      };
      int page1 = -1;
      uint32_t ek1 = 0, ev1 = 0;
      auto read_powers = [&](int page) {  // nothing here waits for what it reads
        ek1 = ev1 = 0;
        if (page < 0 || page >= a.c.num_pages) return;
        const size_t at = static_cast<size_t>(page * a.c.hkv + p.g) * kPage + row % kPage;
        ek1 = a.c.k_scale[at];
        ev1 = a.c.v_scale[at];
      };
      if constexpr (CODES) {
        read_powers(page_id(0));
        page1 = page_id(1);
      }
      int j = 0;
#pragma unroll 1
      for (; j < blks; ++j, ++t) {
        const uint32_t ek = ek1, ev = ev1;
        if constexpr (CODES) {
          read_powers(page1);
          page1 = page_id(j + 2);
        }
        // which columns see this thread's key
        const bool border = (p.blk0 + j + 1) * kBlk > p.len - p.n;
        uint32_t vis = 0xffffffffu;
        if (border) {
          const int key = (p.blk0 + j) * kBlk + row, in_tree = key - (p.len - p.n);
          if (key >= p.len) vis = 0;
          if (key < p.len && in_tree >= 0) {
            const uint32_t* word = a.mask + static_cast<size_t>(p.lo + p.tok0) * a.words + in_tree / 32;
            const int left = p.n - p.tok0, words = a.words;
            vis = 0;
            for (int node0 = c0 / G; node0 * G < c0 + W; node0 += 8) {
              uint32_t m[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) m[i] = node0 + i < left ? word[(node0 + i) * words] : 0u;
              int from = node0 * G - c0;
#pragma unroll
              for (int i = 0; i < 8; ++i, from += G) {
                const int lo = i == 0 ? max(from, 0) : from;
                // its columns, where its bit is set
                vis |= bits_from(lo, from + G - lo) & static_cast<uint32_t>(static_cast<int>(m[i] << (~in_tree & 31)) >> 31);
              }
            }
          }
        }
        if (!wait_warp(sh.s_full, 2, t)) break;
        tc_fence_after();
        const uint32_t s_at = tmem + (t & 1) * N + c0;
        float x[W];
        // scores, less their references where they have one, base 2
        auto scores = [&](bool plain) {
          const float k_factor = CODES ? (ek == 0 ? 1.f : pow2_byte(ek)) : 1.f;
          tmem_ld_cols<W>(s_at, x);
#pragma unroll
          for (int i = 0; i < W; i += 4) {
            const float4 r = plain ? make_float4(0.f, 0.f, 0.f, 0.f) : *reinterpret_cast<const float4*>(&neg_ref[i]);
            float2 f0 = make_float2(a.scale_log2, a.scale_log2), f1 = f0;
            if constexpr (CODES) {
              const float4 f = *reinterpret_cast<const float4*>(&sh.row_factor[c0 + i]);
              const float2 kf = make_float2(k_factor, k_factor);
              f0 = mul2(make_float2(f.x, f.y), kf);
              f1 = mul2(make_float2(f.z, f.w), kf);
            }
            const float2 y0 = fma2(make_float2(x[i], x[i + 1]), f0, make_float2(r.x, r.y));
            const float2 y1 = fma2(make_float2(x[i + 2], x[i + 3]), f1, make_float2(r.z, r.w));
            x[i] = y0.x;
            x[i + 1] = y0.y;
            x[i + 2] = y1.x;
            x[i + 3] = y1.y;
          }
          if (border) {
            asm volatile("");  // a branch, not 32 selections in every block
#pragma unroll
            for (int i = 0; i < W; ++i) x[i] = (vis >> i) & 1 ? x[i] : -INFINITY;
          }
        };
        auto weights = [&]() {
#pragma unroll
          for (int i = 0; i < W; ++i) x[i] = fast_exp2(x[i]);
        };
        // The weights are taken before it is known that no warp has a score past its
        // reference by more than the margin; the rare block that has takes them again.
        bool moves = true;
        if (j > 0) {
          scores(false);
          float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
          for (int i = 4; i + 8 <= W; i += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k) mx[k] = fmaxf(fmaxf(mx[k], x[i + k]), x[i + k + 4]);
#pragma unroll
          for (int k = 0; k < 4; ++k) mx[k] = fmaxf(mx[k], x[W - 4 + k]);
          bool grows = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) > static_cast<float>(C::kMargin);
          if constexpr (CODES) grows = grows || static_cast<int>(ev) > e_ref;
          grows = __any_sync(0xffffffffu, grows);
          if (lane == 0) {
            if (grows) *const_cast<volatile int*>(&sh.moved[wg][t & 1]) = t + 1;
            mbar_arrive(&sh.vote[wg][t & 1]);
          }
          weights();
          if (!wait_warp(sh.vote[wg], 2, t)) break;
          moves = *const_cast<volatile int*>(&sh.moved[wg][t & 1]) == t + 1;
        } else if (lane == 0) {
          mbar_arrive(&sh.vote[wg][t & 1]);
        }
        if (moves) {
          scores(true);
          const float top = over_lanes<W>(x, lane, [](float u, float v) { return fmaxf(u, v); });
          const int turn = syncs & 1;
          if (lane < W) sh.part[wg][turn][quarter][lane] = top;
          if constexpr (CODES) {
            const int e = __reduce_max_sync(0xffffffffu, static_cast<int>(ev));
            if (lane == 0) sh.part_e[wg][turn][quarter] = e;
          }
          if (!sync_warpgroup()) break;
          const auto& of = sh.part[wg][turn];
          const float was = j > 0 ? -neg_ref[c] : -kNone;
          const float now = fmaxf(was, fmaxf(fmaxf(of[0][c], of[1][c]), fmaxf(of[2][c], of[3][c])));
          int e_now = e_ref;
          if constexpr (CODES) {
            const int* e = sh.part_e[wg][turn];
            e_now = max(e_now, max(max(e[0], e[1]), max(e[2], e[3])));
          }
          const float fl = exp2f(was - now), fo = CODES ? fl * pow2_int(e_ref - e_now) : fl;
          e_ref = e_now;
          __syncwarp();
          if (lane < W) neg_ref[lane] = -now;
          __syncwarp();
          if (j > 0) {
#pragma unroll
            for (int i = 0; i < W; i += 2)
              l[i / 2] = mul2(l[i / 2], make_float2(__shfl_sync(0xffffffffu, fl, i), __shfl_sync(0xffffffffu, fl, i + 1)));
            // O holds every product up to the block before once that is done
            if (!wait_warp(sh.p_empty, C::kPBufs, t - 1)) break;
            tc_fence_after();
#pragma unroll 1
            for (int i0 = 0; i0 < W; i0 += 16) {
#pragma unroll 1
              for (int at = 0; at < C::kOCols; at += N) {
                float o[16];
                tmem_ld_cols<16>(o_at + at + i0, o);
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] *= __shfl_sync(0xffffffffu, fo, i0 + i);
                tmem_st_cols<16>(o_at + at + i0, o);
              }
            }
          }
          scores(false);
          weights();
        }
        // The weights' sums, and their terms in the threads' rows of P. Where there are two of
        // it, the product of two blocks ago has read this one: it was issued before these scores.
        if (C::kPBufs == 1 && t >= 1 && !wait_warp(sh.p_empty, 1, t - 1)) break;
        uint8_t* prow = base + C::kOffP + t % C::kPBufs * C::kP + (row >> 3) * 1024 + (row & 7) * 128;
        auto put = [&](int term, int byte, const uint4& v) {  // 16 bytes of the term's columns from `byte` on
          const int at = term * C::kTermBytes + byte;
          *reinterpret_cast<uint4*>(prow + at / 128 * C::kPBlock + ((((at % 128) >> 4) ^ (row & 7)) << 4)) = v;
        };
#pragma unroll
        for (int i = 0; i < W; i += 2) l[i / 2] = add2(l[i / 2], make_float2(x[i], x[i + 1]));
        if constexpr (CODES) {
          const float up = pow2_int(static_cast<int>(ev) - e_ref + C::kLift);
#pragma unroll
          for (int i0 = 0; i0 < W; i0 += 16) {
            uint32_t w[3][4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              // an fp16's upper byte is an e5m2, cut off; what is left is exact in fp16
              uint32_t two[3][2];
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int i = i0 + 4 * k + 2 * h;
                const float2 v = mul2(make_float2(x[i], x[i + 1]), make_float2(up, up));
                __half2 rest = __floats2half2_rn(v.x, v.y);
#pragma unroll
                for (int term = 0; term < 3; ++term) {
                  uint32_t& u = two[term][h];
                  u = *reinterpret_cast<const uint32_t*>(&rest);
                  if (term == 2) {
                    u += 0x00800080u;  // the last one is rounded
                  } else {
                    u &= 0xff00ff00u;
                    rest = __hsub2(rest, *reinterpret_cast<const __half2*>(&u));
                  }
                }
              }
#pragma unroll
              for (int term = 0; term < 3; ++term) w[term][k] = __byte_perm(two[term][0], two[term][1], 0x7531);
            }
#pragma unroll
            for (int term = 0; term < 3; ++term)
              put(term, c0 + i0, make_uint4(w[term][0], w[term][1], w[term][2], w[term][3]));
          }
        } else {
#pragma unroll
          for (int i0 = 0; i0 < W; i0 += 8) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 e = make_float2(x[i0 + 2 * k], x[i0 + 2 * k + 1]);
              if constexpr (C::kTerms == 1) {
                hi[k] = pack_bf16(e.x, e.y);
              } else {
                // the high term cut off, not rounded, and the low one not 0 beside it: an
                // infinite value times both is that infinity, not a NaN
                const uint32_t ux = __float_as_uint(e.x), uy = __float_as_uint(e.y);
                hi[k] = __byte_perm(ux, uy, 0x7632);
                const float2 h = make_float2(__uint_as_float(ux & 0xffff0000u), __uint_as_float(uy & 0xffff0000u));
                const float2 rest = fma2(h, make_float2(-1.f, -1.f), e), least = mul2(h, make_float2(0x1p-30f, 0x1p-30f));
                lo[k] = pack_bf16(fmaxf(rest.x, least.x), fmaxf(rest.y, least.y));
              }
            }
            put(0, 2 * (c0 + i0), make_uint4(hi[0], hi[1], hi[2], hi[3]));
            if constexpr (C::kTerms == 2) put(1, 2 * (c0 + i0), make_uint4(lo[0], lo[1], lo[2], lo[3]));
          }
        }
        // Value rows past the sequence's end (the tail of the last page, pages not loaded) are
        // zeroed: what their slots hold must not reach O as 0 * NaN.
        if (wg == 0 && (p.blk0 + j + 1) * kBlk > p.len) {
          if (!wait_warp(sh.v_full, C::kDepth, t)) break;
          if ((p.blk0 + j) * kBlk + row >= p.len) {
            uint8_t* v = base + C::kOffV + t % C::kDepth * C::kSlot + row * 128;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              *reinterpret_cast<uint4*>(v + 16 * i) = make_uint4(0u, 0u, 0u, 0u);
              if constexpr (!CODES) *reinterpret_cast<uint4*>(v + C::kHalf + 16 * i) = make_uint4(0u, 0u, 0u, 0u);
            }
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        // P is there, and the scores have been read: two blocks on they are written over, behind
        // the product that waits for this
        if (lane == 0) mbar_arrive(&sh.p_full[t % C::kPBufs]);
      }
      if (j < blks) break;  // a wait has failed
      // ---- the piece's rows: the sums over the keys, then O, column by column
      float x[W];
#pragma unroll
      for (int i = 0; i < W; i += 2) {
        x[i] = l[i / 2].x;
        x[i + 1] = l[i / 2].y;
      }
      const float of_warp = over_lanes<W>(x, lane, [](float u, float v) { return u + v; });
      const int turn = syncs & 1;
      if (lane < W) sh.part[wg][turn][quarter][lane] = of_warp;
      if (!sync_warpgroup()) break;
      const auto& of = sh.part[wg][turn];
      const float sum = (of[0][c] + of[1][c]) + (of[2][c] + of[3][c]);
      const float ref = -neg_ref[c];
      // no key seen (scores that are all NaN move no reference either)
      const bool none = ref == -kNone && sum == 0.f;
      const int slot = p.slot;
      const size_t part = (static_cast<size_t>(blockIdx.x) * 2 + max(slot, 0)) * N + c0;
      // every column's row and factor, for all lanes
      auto* last = sh.last[wg][quarter];
      if (lane < W) {
        last[lane].row = c_row;
        last[lane].factor = none ? 0.f : (CODES ? 1.f / static_cast<float>(1 << C::kLift) : 1.f) / sum;
      }
      const float f2 = CODES ? pow2_int(e_ref - 127) : 1.f;
      __syncwarp();
      if (!wait_warp(sh.p_empty, C::kPBufs, t - 1)) break;
      tc_fence_after();
      bf16* out = a.out + row;
      float* out_part = a.part_o + part * 128 + row;
#pragma unroll 1
      for (int i0 = 0; i0 < W; i0 += 16) {  // 16 columns at a time: the code runs once a piece, and is fetched for it
        float o[16];
        tmem_ld_cols<16>(o_at + i0, o);
#pragma unroll 1
        for (int at = N; at < C::kOCols; at += N) {
          float more[16];
          tmem_ld_cols<16>(o_at + at + i0, more);
#pragma unroll
          for (int i = 0; i < 16; ++i) o[i] += more[i];
        }
        if (slot < 0) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int r = last[i0 + i].row;
            const float fi = last[i0 + i].factor;
            if (r >= 0) out[static_cast<size_t>(r) * 128] = __float2bfloat16(fi == 0.f ? 0.f : o[i] * fi * f2);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (last[i0 + i].row >= 0) out_part[(i0 + i) * 128] = o[i];
        }
      }
      if (quarter == 0 && lane < W && c_there) {
        if (slot >= 0)
          a.part_st[part + lane] = none ? PartStat{-INFINITY, -INFINITY, 0.f, 0.f}
                                        : PartStat{CODES ? ref + static_cast<float>(e_ref - 127 - C::kLift) : ref, ref, sum, 0.f};
        else if (a.lse != nullptr)
          a.lse[c_row] = none ? -INFINITY : (ref + log2f(sum)) * 0.6931471805599453f;
      }
      tc_fence_before();
      done_piece();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(sh.tmem, C::kTmem);
  }
  if (threadIdx.x == 0 && *abort_flag) raise_device_error(a.c.err, QUAIL_ERR_DEVICE_TIMEOUT, 6000);
}

// ------------------------------------------------------------------ join
// Rows whose item several CTAs shared: the part of the one that began it (slot 0 of its
// two), then those of the CTAs after it (slot 1), brought to one maximum. A block for 8
// columns of a CTA's item, a warp a row, 4 dims a lane; most find that their CTA left
// none. And the rows of sequences without keys, which are in no CTA's work.
constexpr int kJoinWarps = 8;
__global__ void __launch_bounds__(32 * kJoinWarps) tree_join_kernel(TreeAttnArgs a) {
  grid_dependency_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, G = a.hq / a.c.hkv;
  if (blockIdx.y == 0) {
    for (int b0 = 32 * (blockIdx.x * kJoinWarps + warp); b0 < a.c.num_seqs; b0 += 32 * kJoinWarps * gridDim.x) {
      const Seq mine = b0 + lane < a.c.num_seqs ? seq_of(a, b0 + lane) : Seq{0, 0, 0, false};
      for (uint32_t empty = __ballot_sync(0xffffffffu, mine.ok && mine.len == 0 && mine.n > 0); empty != 0; empty &= empty - 1) {
        const int from = __ffs(empty) - 1;
        const size_t row0 = static_cast<size_t>(__shfl_sync(0xffffffffu, mine.lo, from)) * a.hq;
        const int rows = __shfl_sync(0xffffffffu, mine.n, from) * a.hq;
        for (int i = lane; i < rows * 16; i += 32) reinterpret_cast<uint4*>(a.out + row0 * 128)[i] = make_uint4(0u, 0u, 0u, 0u);
        for (int i = lane; a.lse != nullptr && i < rows; i += 32) a.lse[row0 + i] = -INFINITY;
      }
    }
  }
  const SharedItem it = a.shared_items[blockIdx.x];
  const int col = blockIdx.y * kJoinWarps + warp;
  if (it.parts < 2 || col >= it.tokens * G) return;
  const size_t row = static_cast<size_t>(it.row0 + col / G) * a.hq + it.g * G + col % G;
  auto at = [&](int i) { return (static_cast<size_t>(blockIdx.x + i) * 2 + (i > 0)) * a.tile_cols + col; };
  PartStat st{-INFINITY, -INFINITY, 0.f, 0.f};
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  auto pow2_or_0 = [](float x, float ref) { return x == -INFINITY ? 0.f : exp2f(x - ref); };
  for (int i0 = 0; i0 < it.parts; i0 += 32) {
    const int n = min(32, it.parts - i0);
    const PartStat mine = lane < n ? a.part_st[at(i0 + lane)] : PartStat{-INFINITY, -INFINITY, 0.f, 0.f};
    float mo = fmaxf(mine.m_o, st.m_o), ml = fmaxf(mine.m_l, st.m_l);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      mo = fmaxf(mo, __shfl_xor_sync(0xffffffffu, mo, d));
      ml = fmaxf(ml, __shfl_xor_sync(0xffffffffu, ml, d));
    }
    const float f = pow2_or_0(mine.m_o, mo), was = pow2_or_0(st.m_o, mo);
    float l = mine.l != mine.l ? mine.l : mine.l * pow2_or_0(mine.m_l, ml);  // a NaN sum stays one
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
    acc = make_float4(acc.x * was, acc.y * was, acc.z * was, acc.w * was);
    st.l = (st.l != st.l ? st.l : st.l * pow2_or_0(st.m_l, ml)) + l;
    st.m_l = ml;
    st.m_o = mo;
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      const float4 v = *reinterpret_cast<const float4*>(a.part_o + at(i0 + i) * 128 + 4 * lane);
      const float w = __shfl_sync(0xffffffffu, f, i);
      acc = make_float4(fmaf(v.x, w, acc.x), fmaf(v.y, w, acc.y), fmaf(v.z, w, acc.z), fmaf(v.w, w, acc.w));
    }
  }
  const bool none = st.m_l == -INFINITY && st.l == 0.f;
  const float f = none ? 0.f : st.l != st.l ? st.l : exp2f(st.m_o - st.m_l) / st.l;
  if (none) acc = make_float4(0.f, 0.f, 0.f, 0.f);  // whatever weights of 0 made of the values
  *reinterpret_cast<uint2*>(a.out + row * 128 + 4 * lane) =
      make_uint2(pack_bf16(acc.x * f, acc.y * f), pack_bf16(acc.z * f, acc.w * f));
  if (lane == 0 && a.lse != nullptr) a.lse[row] = none ? -INFINITY : (st.m_l + log2f(st.l)) * 0.6931471805599453f;
}

template <int N, bool CODES>
cudaError_t launch(const TreeAttnArgs& a, const CUtensorMap& tmK, const CUtensorMap& tmV, const CUtensorMap& tmQ, int ctas,
                   cudaStream_t st) {
  auto kern = tree_attention_kernel<N, CODES>;
  constexpr size_t smem = tree_smem<N, CODES>();
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
  return launch_pdl(kern, dim3(ctas), dim3(Cfg<N, CODES>::kThreads), smem, st, a, tmK, tmV, tmQ);
}

}  // namespace

cudaError_t launch_tree_attention(const TreeAttnArgs& a, const CUtensorMap& tmK, const CUtensorMap& tmV,
                                  const CUtensorMap& tmQ, cudaStream_t st) {
  cudaError_t e;
  const auto go = [&](auto cols) {
    constexpr int kN = decltype(cols)::value;
    return a.c.codes ? launch<kN, true>(a, tmK, tmV, tmQ, a.ctas, st) : launch<kN, false>(a, tmK, tmV, tmQ, a.ctas, st);
  };
  switch (a.tile_cols) {
    case 16: e = go(std::integral_constant<int, 16>{}); break;
    case 32: e = go(std::integral_constant<int, 32>{}); break;
    case 64: e = go(std::integral_constant<int, 64>{}); break;
    case 96: e = go(std::integral_constant<int, 96>{}); break;
    default: e = go(std::integral_constant<int, 128>{}); break;
  }
  if (e != cudaSuccess || a.direct) return e;
  count_launch();
  return launch_pdl(tree_join_kernel, dim3(a.ctas, a.tile_cols / kJoinWarps), dim3(32 * kJoinWarps), 0, st, a);
}

// Test hook: this translation unit's copy of the pipeline wait limit.
cudaError_t set_pipeline_wait_limit_tree_attention(long long cycles) {
  return cudaMemcpyToSymbol(g_pipeline_wait_limit, &cycles, sizeof(cycles));
}

}  // namespace quail
