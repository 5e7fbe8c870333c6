// Attention over the paged document cache on tcgen05, for many query rows per
// KV head. Two uses of one kernel:
//   shared prefix -- the rows of every sequence of the batch side by side, so
//                    the prefix keys are read and multiplied once for all;
//   sequences     -- a sequence's own rows over its keys (all of them, or those
//                    past the prefix), each row up to its causal limit.
// A CTA owns 256 query rows as two 128-row tiles that share every K and V
// block of 128 keys (8 pages):
//   S_t = Q_t K^T   M 128, N 128 keys, K 128 dims; Q_t and K in shared memory
//   O_t += P_t V    M 128, N 128 dims, K 128 keys; P_t (bf16) in TMEM over S_t
// with fp32 S and O in TMEM (2 x (128 + 128) columns, all 512). The issue order
// PV_0(j) S_0(j+1) PV_1(j) S_1(j+1) keeps the tensor pipe on one tile while the
// softmax warpgroup of the other works. The four products of a block are 2,048
// tensor cycles; with the softmax between them a block takes 2,800 to 3,150, since
// S -> maximum -> weights -> P of a tile (1,630, a thread to a row) and its own two
// products (1,024) are one chain: the tensor memory has no room for a second S. A CTA takes another 3,000
// to 5,000 to its first S and 3,000 to write its rows.
// 16 prefills of 128 to 1,024 tokens behind 2,048 (32 heads on 8): 318 us,
// 1,160 TFLOP/s. A CTA with one tile's rows is bound by that
// tile's chain, 1.45 us a block; e4m3 1.9 us, the widening warps competing with it
// for shared memory.
//
// P is one bf16 term, so o is off by 0.0023 relative where its own rounding alone gives
// 0.0017. A second term in the other half of S's columns gives that 0.0017 and costs half
// as many products again (3,072 clocks a block); written the plain way, which spills 650 to
// 800 bytes, the 16 prefills took 732 us.
//
// The softmax keeps 128 scores, 32 columns of P and its sums in 200 registers, and spills a
// little for it: 32 and 44 bytes (bf16), 120 and 136 (e4m3, launched with 128).
//
// Few CTAs' worth of rows: their keys are cut into up to eight ranges, a CTA each in one
// cluster, which leave their parts in shared memory and join them there row by row
// (more ranges, and parts of other kernels, go through memory and the join kernel).
//
// Roles (384 threads, over codes 512): warps 0 and 3 load K and V pages into one ring
// K0 V0 K1 V1 .., warp 1 owns TMEM and issues the MMAs (a second issuer, one for each
// tile, let the tiles' MMAs interleave and was slower), warps 4-7 and 8-11 are the
// softmax of tile 0 and 1, one thread per row (no exchange between threads),
// which also load their Q rows and write their O rows. Over an e4m3 cache the loaders
// fill a ring of codes (half the bytes) and warps 12-15 (with an empty second tile
// 8-11 too) widen each block, times its rows' powers of two, into the ring of bf16
// that the MMAs read: exact, so a code takes part as the bf16 value that it stands for.
#include <atomic>

#include "cache_attn.cuh"
#include "launch.cuh"

namespace quail {

namespace {

constexpr int kBlkKeys = 128;
constexpr int kBlkPages = kBlkKeys / kPage;
constexpr uint32_t kHalf = kBlkKeys * 128;  // 128 rows x 64 bf16, 128-byte rows, swizzled
constexpr uint32_t kStage = 2 * kHalf;
constexpr uint32_t kOffQ = 0;  // two tiles
constexpr uint32_t kOffRing = 2 * kStage;
constexpr uint32_t kTmemO = 256;
constexpr int kSoftmaxRegs = 200;  // the softmax keeps a whole row of S

template <bool CODES>
struct TileCfg {
  static constexpr int kThreads = CODES ? 512 : 384;
  static constexpr int kStages = CODES ? 3 : 5;      // blocks of K or V that the MMAs read
  static constexpr int kCodeStages = CODES ? 4 : 0;  // blocks of codes on their way
  static constexpr uint32_t kCodeStage = kBlkKeys * 128;
  static constexpr uint32_t kOffCodes = kOffRing + kStages * kStage;
  static constexpr uint32_t kOffScales = kOffCodes + kCodeStages * kCodeStage;
  static constexpr uint32_t kOffBar = kOffScales + kCodeStages * kBlkKeys;
  // registers a thread: at launch, and of the warps beside the softmax's 256 threads
  static constexpr int kLaunchRegs = CODES ? 128 : 168, kOtherRegs = CODES ? 56 : 104;
  static_assert(256 * kSoftmaxRegs + (kThreads - 256) * kOtherRegs <= kThreads * kLaunchRegs,
                "the split draws on the launch's registers");
};

struct Bars {
  uint64_t full[5], empty[5];
  uint64_t code_full[4], code_empty[4];
  uint64_t s_full[2], p_full[2], pv_done[2], q_full, drain;
  uint32_t tmem_slot;
  int abort_flag;
};
template <bool CODES>
constexpr size_t tile_smem() {
  constexpr size_t n = 1024 + TileCfg<CODES>::kOffBar + sizeof(Bars);
  static_assert(n <= 227 * 1024, "shared memory");
  return n;
}

// Starts the load of 32 columns; the registers hold them after tmem_ld_wait,
// which names them so that no use can move ahead of it.
__device__ __forceinline__ void tmem_ld_32cols_nowait(uint32_t taddr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      :
        "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
        "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]),
        "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]),
        "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               :
        "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]),
        "+r"(v[7]), "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]),
        "+r"(v[14]), "+r"(v[15]), "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]),
        "+r"(v[21]), "+r"(v[22]), "+r"(v[23]), "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]),
        "+r"(v[28]), "+r"(v[29]), "+r"(v[30]), "+r"(v[31])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_st_32cols_nowait(uint32_t taddr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
      "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
      "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}
// 16 columns, waited for.
__device__ __forceinline__ void tmem_ld_16cols(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st_16cols(uint32_t taddr, const float (&v)[16]) {
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

// The tensor memory that warp 1 has taken, for it and the softmax warps.
__device__ __forceinline__ uint32_t tmem_ready(const Bars* bars) {
  tc_fence_before();
  asm volatile("bar.sync 1, 288;" ::: "memory");
  tc_fence_after();
  return bars->tmem_slot;
}

// 16 bytes, or two floats, at this CTA's shared address `at` in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t in_cta(uint32_t at, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(at), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t at) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ float2 ld_cluster2(uint32_t at) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
  return v;
}
// A clustered CTA's part: 256 rows of 128 fp32, chunk c of row r at (c ^ (r & 7)),
// then their (maximum, sum). It lies over the queries and the rings.
__device__ __forceinline__ uint32_t part_at(int row, int chunk) { return row * 512u + ((chunk ^ (row & 7)) << 4); }
constexpr uint32_t kPartStats = kTileRows * 512;
static_assert(kPartStats + kTileRows * 8 <= TileCfg<false>::kOffBar && kPartStats + kTileRows * 8 <= TileCfg<true>::kOffBar,
              "a part fits over the queries and the rings");

struct Item {
  int row0, n_rows;  // this CTA's first row and the rows there are, per KV head
  int k_lo, k_hi;    // keys
  int b;             // sequence, or -1: the shared prefix for all rows
  int g, split;
};

// Eight codes times 2^(e - 127) as bf16. A code's magnitude bits, moved to bits 4-10
// of a bf16, are its value times 2^-120 (its subnormals too), so one product with
// m2 = (2^(e - 7), 2^(e - 7)) finishes a pair: a byte permute that extends the signs,
// a product by 16, a mask and a bf16 product.
__device__ __forceinline__ uint4 widen8(uint32_t a, uint32_t b, uint32_t m2) {
  const uint32_t w[2] = {a, b};
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t y;  // two bytes as signed 16-bit numbers
    asm("prmt.b32 %0, %1, 0, %2;" : "=r"(y) : "r"(w[i >> 1]), "r"((i & 1) == 0 ? 0x9180 : 0xb3a2));
    y = y * 16u & 0x87f087f0u;
    const __nv_bfloat162 v =
        __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&y), *reinterpret_cast<const __nv_bfloat162*>(&m2));
    r[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}
// The same for any code and e, NaN and scales from 2^8 on included, by conversions.
__device__ __forceinline__ uint4 widen8_any(uint32_t a, uint32_t b, float f) {
  uint32_t h[4], r[4];
  widen4(a, h[0], h[1]);
  widen4(b, h[2], h[3]);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    r[i] = pack_bf16(v.x * f, v.y * f);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// Blocks first, first + step, .. of the code ring (K0 V0 K1 V1 ..) into the ring that
// the MMAs read; warp w of four takes 32 rows of each. Eight lanes to a row of 128
// codes, 16 each: two 16-byte chunks of bf16. Lanes of a row's second half store
// theirs in the other order, so that eight lanes always hit eight different chunks
// of a row's 128 bytes. A warp whose rows hold a NaN or a large scale, or rows past
// the range, does them again the long way: the loop that all others take has no
// branch (2,400 clocks a block with one, 1,750 without).
__device__ __forceinline__ void widen_blocks(uint8_t* base, Bars* bars, int w, int lane, int first, int step,
                                             int n_blocks, int n_keys, long long limit_clk) {
  using Cfg = TileCfg<true>;
  volatile int* abort_flag = &bars->abort_flag;
  const int c = lane & 7, half = c >> 2, ch = 2 * (c & 3) + half;
  for (int idx = first; idx < 2 * n_blocks; idx += step) {
    const int cs = idx % Cfg::kCodeStages, s = idx % Cfg::kStages, use = idx / Cfg::kStages;
    const bool here =
        wait_bar(&bars->code_full[cs], static_cast<uint32_t>((idx / Cfg::kCodeStages) & 1), abort_flag, limit_clk) &&
        (use == 0 || wait_bar(&bars->empty[s], static_cast<uint32_t>((use - 1) & 1), abort_flag, limit_clk));
    if (!__all_sync(0xffffffffu, here)) break;
    const uint8_t* code = base + Cfg::kOffCodes + cs * Cfg::kCodeStage;
    const uint8_t* exps = base + Cfg::kOffScales + cs * kBlkKeys;
    uint8_t* dst = base + kOffRing + s * kStage + half * kHalf;
    uint32_t odd = 0;
    auto row_of = [&](int i) { return 32 * w + 4 * i + (lane >> 3); };
#pragma unroll 2
    for (int i = 0; i < 8; ++i) {
      const int row = row_of(i), sw = row & 7;
      const uint4 x = *reinterpret_cast<const uint4*>(code + row * 128 + ((c ^ sw) << 4));
      const uint32_t e = exps[row], m = (e + 120) << 7;
      odd |= ((x.x & 0x7f7f7f7fu) + 0x01010101u) | ((x.y & 0x7f7f7f7fu) + 0x01010101u);
      odd |= ((x.z & 0x7f7f7f7fu) + 0x01010101u) | ((x.w & 0x7f7f7f7fu) + 0x01010101u);
      odd |= (e + 121) >> 1 & 0x80u;  // e > 134: 2^(e - 7) is no bf16
      const uint32_t m2 = m | m << 16;
      *reinterpret_cast<uint4*>(dst + row * 128 + ((ch ^ sw) << 4)) = widen8(half ? x.z : x.x, half ? x.w : x.y, m2);
      *reinterpret_cast<uint4*>(dst + row * 128 + (((ch ^ 1) ^ sw) << 4)) = widen8(half ? x.x : x.z, half ? x.y : x.w, m2);
    }
    // value rows past the range are zeros, whatever their slots hold
    const int rows = (idx & 1) ? n_keys - (idx >> 1) * kBlkKeys : kBlkKeys;
    if (__any_sync(0xffffffffu, (odd & 0x80808080u) != 0) || rows < 32 * (w + 1)) {
#pragma unroll 1
      for (int i = 0; i < 8; ++i) {
        const int row = row_of(i), sw = row & 7;
        uint4 x = *reinterpret_cast<const uint4*>(code + row * 128 + ((c ^ sw) << 4));
        const float f = row < rows ? pow2_byte(exps[row]) : 0.f;
        if (row >= rows) x = make_uint4(0u, 0u, 0u, 0u);
        *reinterpret_cast<uint4*>(dst + row * 128 + ((ch ^ sw) << 4)) = widen8_any(half ? x.z : x.x, half ? x.w : x.y, f);
        *reinterpret_cast<uint4*>(dst + row * 128 + (((ch ^ 1) ^ sw) << 4)) = widen8_any(half ? x.x : x.z, half ? x.y : x.w, f);
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(&bars->code_empty[cs]);
      mbar_arrive(&bars->full[s]);
    }
  }
}

template <bool PREFIX, bool CODES>
__global__ void __launch_bounds__(TileCfg<CODES>::kThreads, 1)
    attention_tile_kernel(SharedAttnArgs a, const __grid_constant__ CUtensorMap tmK,
                          const __grid_constant__ CUtensorMap tmV) {
  using Cfg = TileCfg<CODES>;
  constexpr int kThreads = Cfg::kThreads, kStages = Cfg::kStages;
  extern __shared__ uint8_t smem_raw[];
  // by an offset: from an address rounded up, the compiler could not tell shared memory
  uint8_t* base = smem_raw + (-smem_u32(smem_raw) & 1023u);
  Bars* bars = reinterpret_cast<Bars*>(base + Cfg::kOffBar);
  volatile int* abort_flag = &bars->abort_flag;
  const long long limit_clk = pipeline_wait_limit();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.hq / a.c.hkv;
  // Behind the streaming kernel (prefix tiles only, no early exit) nothing here
  // depends on it: it lets this kernel launch after its own wait, so all that
  // came before it is complete, and these CTAs start on the SMs that it leaves
  // first, 20 to 30 us before its last. The wait then comes before the exit.
  const bool behind_stream = PREFIX && a.streamed;
  if (!behind_stream) grid_dependency_wait();
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bars->full[s], CODES ? 4 : 1);  // the warps that widen, or the loader
      mbar_init(&bars->empty[s], 1);
    }
    for (int s = 0; s < Cfg::kCodeStages; ++s) {
      mbar_init(&bars->code_full[s], 1 + kBlkPages);  // the loader, and its lanes' copies of exponents
      mbar_init(&bars->code_empty[s], 4);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bars->s_full[t], 1 + (limit_clk < 0));
      mbar_init(&bars->p_full[t], 128);
      mbar_init(&bars->pv_done[t], 1);
    }
    mbar_init(&bars->q_full, 256);
    mbar_init(&bars->drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();

  Item it;
  QueryRange qr{0, 0, 0, true};
  int first_page = -1;  // of a loader's lane, asked for along with the lengths that say whether it is in range
  it.g = blockIdx.y;
  if constexpr (PREFIX) {
    it.b = -1;
    it.row0 = blockIdx.x * kTileRows;
    it.n_rows = a.total_q * G;
    it.split = blockIdx.z;
    it.k_lo = it.split * a.prefix_split;
    it.k_hi = min(a.prefix_len, it.k_lo + a.prefix_split);
    if (warp < 4 && it.k_lo / kPage + lane < a.prefix_len / kPage) first_page = a.prefix_pages[it.k_lo / kPage + lane];
  } else {
    // the rows that see the most keys first
    it.b = blockIdx.z;
    it.split = blockIdx.x % a.seq_splits;
    it.row0 = (gridDim.x / a.seq_splits - 1 - blockIdx.x / a.seq_splits) * kTileRows;
    it.k_lo = a.seq_begin + it.split * a.seq_split;
    if (warp < 4) {
      const int p = it.k_lo / kPage + lane;
      if (p < a.prefix_len / kPage)
        first_page = a.prefix_pages[p];
      else if (p < a.c.max_pages)
        first_page = a.c.table[static_cast<size_t>(it.b) * a.c.max_pages + p];
    }
    qr = query_range(a, it.b);
    if (!qr.ok) {
      if (threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0)
        raise_device_error(a.c.err, QUAIL_ERR_DEVICE_BOUNDS, it.b);
      return;
    }
    it.n_rows = (qr.hi - qr.lo) * G;
    if (it.row0 >= it.n_rows) return;
    if (qr.len == 0) {  // no key: zeros, here or in the join
      if (a.dense_parts == 0) {
        for (int i = threadIdx.x; i < min(kTileRows, it.n_rows - it.row0) * 16; i += kThreads) {
          const int r = it.row0 + i / 16;
          const size_t row = static_cast<size_t>(qr.lo + r / G) * a.hq + it.g * G + r % G;
          reinterpret_cast<uint4*>(a.out + row * 128)[i % 16] = make_uint4(0u, 0u, 0u, 0u);
          if (i % 16 == 0 && a.lse != nullptr) a.lse[row] = -INFINITY;
        }
      }
      return;
    }
    it.k_hi = min(tile_key_end(a, qr, it.row0), it.k_lo + a.seq_split);
    if (it.k_hi <= it.k_lo) {  // no key of these rows' in this range
      if (a.clustered) {
        cluster_sync();
        cluster_sync();
      }
      return;
    }
  }
  const bool two = it.n_rows - it.row0 > 128;
  const int n_pages = (it.k_hi - it.k_lo + kPage - 1) / kPage;
  const int n_blocks = (n_pages + kBlkPages - 1) / kBlkPages;

  // Query rows of the softmax warps: a warp's 32 rows, half a warp to a row of 256 bytes. Rows past the last
  // read the first one, and nothing reads theirs; asking for each row made the loads
  // wait for one another, 7,000 clocks a CTA.
  const int t = (warp - 4) >> 2, quarter = warp & 3;  // tile and 32-row quarter of a softmax warp
  const int rr = it.row0 + t * 128 + quarter * 32 + lane;  // row of the item
  const bool softmax_warp = warp >= 4 && warp < 12;
  const bool row_ok = softmax_warp && rr < it.n_rows;
  const size_t out_row =
      row_ok ? static_cast<size_t>(qr.lo + rr / G) * a.hq + it.g * G + rr % G : 0;  // (token, head)
  uint4 qx[16];
  if (softmax_warp && (t == 0 || two)) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int row = 2 * i + (lane >> 4);
      const size_t src = __shfl_sync(0xffffffffu, static_cast<unsigned long long>(out_row), row);
      qx[i] = reinterpret_cast<const uint4*>(a.q + src * 128)[lane & 15];
    }
  }

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Cfg::kOtherRegs));
    if (warp == 0 || warp == 3) {
      // ---------------------------------------------- loaders (K: warp 0, V: warp 3)
      // Lane q takes page q of a block; the ids of the next block are read while
      // this one waits for its stage.
      const int kv = warp == 0 ? 0 : 1;
      const CUtensorMap* tm = kv == 0 ? &tmK : &tmV;
      constexpr int kIn = CODES ? Cfg::kCodeStages : kStages;
      uint64_t* full = CODES ? bars->code_full : bars->full;
      uint64_t* empty = CODES ? bars->code_empty : bars->empty;
      const int p0 = it.k_lo / kPage, pp = a.prefix_len / kPage;
      auto page_id = [&](int blk) {
        const int p = p0 + blk * kBlkPages + lane;
        if (lane >= kBlkPages || blk * kBlkPages + lane >= n_pages) return -1;
        return p < pp ? a.prefix_pages[p] : a.c.table[static_cast<size_t>(it.b) * a.c.max_pages + p];
      };
      int next = lane < min(kBlkPages, n_pages) ? first_page : -1, issued = 0;
      for (int blk = 0; blk < n_blocks; ++blk) {
        int page = next;
        if (blk + 1 < n_blocks) next = page_id(blk + 1);
        const bool mine = lane < min(kBlkPages, n_pages - blk * kBlkPages);
        if (mine && (page < 0 || page >= a.c.num_pages)) {
          raise_device_error(a.c.err, QUAIL_ERR_DEVICE_BOUNDS, PREFIX ? 0 : it.b);
          page = -1;  // not copied: the stage's old contents are consumed, the rows are void
        }
        const uint32_t good = __popc(__ballot_sync(0xffffffffu, page >= 0));
        const int idx = 2 * blk + kv, s = idx % kIn, use = idx / kIn;
        if (use > 0 && !__all_sync(0xffffffffu, wait_bar(&empty[s], static_cast<uint32_t>((use - 1) & 1), abort_flag, limit_clk)))
          break;
        if (lane == 0) {
          if (good > 0)
            mbar_arrive_expect_tx(&full[s], good * (CODES ? 2048 : 4096));
          else
            mbar_arrive(&full[s]);
        }
        __syncwarp();
        const int y = (page * a.c.hkv + it.g) * kPage;
        if (page >= 0) {
          if constexpr (CODES) {
            tma_load_2d(base + Cfg::kOffCodes + s * Cfg::kCodeStage + lane * 2048, tm, &full[s], 0, y);
            copy16_async(smem_u32(base + Cfg::kOffScales + s * kBlkKeys + lane * kPage),
                         (kv == 0 ? a.c.k_scale : a.c.v_scale) + static_cast<size_t>(y));
          } else {
            uint8_t* dst = base + kOffRing + s * kStage + lane * 2048;
            tma_load_2d(dst, tm, &full[s], 0, y);
            tma_load_2d(dst + kHalf, tm, &full[s], 64, y);
          }
        }
        if (CODES && lane < kBlkPages) arrive_after_copies(&full[s]);
        ++issued;
      }
      // No copy may still be landing when the CTA exits: wait for this loader's last
      // uses of the stages, but not for one that a later use has followed (a stage is
      // filled again only once it was consumed).
      for (int blk = max(0, issued - (CODES ? 2 : 3)); lane == 0 && blk < issued; ++blk) {
        const int idx = 2 * blk + kv;
        if (issued == n_blocks && idx + kIn < 2 * n_blocks) continue;
        const long long t0 = clock64();
        while (!mbar_try_wait(smem_u32(&full[idx % kIn]), static_cast<uint32_t>((idx / kIn) & 1))) {
          if (clock64() - t0 > kWaitLimitCycles) {
            *abort_flag = 1;
            break;
          }
        }
      }
    } else if (warp == 1) {
      // ---------------------------------------------- MMA issuer
      tmem_alloc(&bars->tmem_slot, 512);
      tmem_relinquish();
      const uint32_t tmem_base = tmem_ready(bars);
      if (lane == 0) {
        constexpr uint32_t idesc_s = umma_idesc_bf16_f32(128, kBlkKeys);
        constexpr uint32_t idesc_pv = umma_idesc_bf16_f32_bmn(128, 128);
        const uint64_t dq = smem_desc_sw128(smem_u32(base + kOffQ));
        const uint64_t dk = smem_desc_sw128(smem_u32(base + kOffRing));
        const uint64_t dv = smem_desc_sw128_mn(smem_u32(base + kOffRing), kHalf, 1024);
        const uint32_t dv_lo = static_cast<uint32_t>(dv), dv_hi = static_cast<uint32_t>(dv >> 32);
        auto wait_full = [&](int idx) {
          return wait_bar(&bars->full[idx % kStages], static_cast<uint32_t>((idx / kStages) & 1), abort_flag, limit_clk);
        };
        auto issue_s = [&](int t, int j) {
          const uint64_t k = dk + (((2 * j) % kStages * kStage) >> 4), q = dq + ((t * kStage) >> 4);
#pragma unroll
          for (int ks = 0; ks < 8; ++ks) {
            const uint32_t off = ((ks >> 2) * kHalf + (ks & 3) * 32) >> 4;
            umma_bf16(tmem_base + t * 128, q + off, k + off, idesc_s, ks != 0 ? 1u : 0u);
          }
          umma_commit(&bars->s_full[t]);
        };
        auto issue_pv = [&](int t, int j) {
          const uint32_t v = dv_lo + (((2 * j + 1) % kStages * kStage) >> 4);
          if (!wait_bar(&bars->p_full[t], static_cast<uint32_t>(j & 1), abort_flag, limit_clk)) return false;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)  // 16 keys = one page per instruction
            umma_ts(tmem_base + kTmemO + t * 128, tmem_base + t * 128 + kk * 8, v + ((kk * 2048) >> 4), dv_hi, idesc_pv,
                    (j > 0 || kk > 0) ? 1u : 0u);
          umma_commit(&bars->pv_done[t]);
          return true;
        };
        bool ok = wait_bar(&bars->q_full, 0u, abort_flag, limit_clk) && wait_full(0);
        if (ok) {
          tc_fence_after();
          issue_s(0, 0);
          if (two) issue_s(1, 0);
          umma_commit(&bars->empty[0]);
        }
        for (int j = 0; ok && j < n_blocks; ++j) {
          const bool more = j + 1 < n_blocks;
          // the pages first: they are there long before the weights (widened ones may
          // not be, and the next keys wait for this product to free their stage)
          ok = wait_full(2 * j + 1) && (CODES || !more || wait_full(2 * j + 2)) && issue_pv(0, j) &&
               (!CODES || !more || wait_full(2 * j + 2));
          if (!ok) break;
          if (CODES) tc_fence_after();
          if (more) issue_s(0, j + 1);
          if (two) {
            ok = issue_pv(1, j);
            if (!ok) break;
          }
          umma_commit(&bars->empty[(2 * j + 1) % kStages]);
          if (more) {
            if (two) issue_s(1, j + 1);
            umma_commit(&bars->empty[(2 * j + 2) % kStages]);
          }
        }
        // every MMA of this thread completes before TMEM is released
        umma_commit(&bars->drain);
        const long long t0 = clock64();
        while (!mbar_try_wait(smem_u32(&bars->drain), 0u)) {
          if (clock64() - t0 > kWaitLimitCycles) {
            *abort_flag = 1;
            break;
          }
        }
      }
    }
  } else if (warp < 12) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ------------------------------------------------ softmax: thread <-> row of tile t
    const int r = quarter * 32 + lane;  // row of the tile = TMEM lane
    uint8_t* q_tile = base + kOffQ + t * kStage;
    if (t == 0 || two) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int row = quarter * 32 + 2 * i + (lane >> 4), c = lane & 15;
        *reinterpret_cast<uint4*>(q_tile + (c >> 3) * kHalf + row * 128 + (((c & 7) ^ (row & 7)) << 4)) = qx[i];
      }
      fence_proxy_async_smem();
    }
    mbar_arrive(&bars->q_full);
    const uint32_t tmem_base = tmem_ready(bars);
    const uint32_t lane_addr = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
    if (t == 0 || two) {
      const int limit = PREFIX || !row_ok ? it.k_hi : min(it.k_hi, row_limit(a, qr, rr));
      // a warp without a row takes part in the waits and leaves its weights as they are
      const bool live = it.row0 + t * 128 + quarter * 32 < it.n_rows;
      const float scale = a.scale_log2;
      float m_ref = -INFINITY, l = 0.f;
      bool ok = true;
      // Keys past the range (tail of the last page, pages not loaded): their V
      // rows are zeroed, so that what the slots hold cannot reach O as 0 * NaN.
      // Tile 0 does it for both: its product is issued first. (Codes are zeroed as
      // they are widened.)
      auto clear_tail = [&](int j, int key0) {
        const int in_range = it.k_hi - key0;
        if (CODES || t != 0 || in_range >= kBlkKeys) return true;
        const int idx = 2 * j + 1;
        if (!__all_sync(0xffffffffu, wait_bar(&bars->full[idx % kStages], static_cast<uint32_t>((idx / kStages) & 1), abort_flag, limit_clk)))
          return false;
        uint8_t* v = base + kOffRing + (idx % kStages) * kStage;
        for (int i = r; i < (kBlkKeys - in_range) * 16; i += 128) {
          const int row = in_range + i / 16, c = i % 16;
          *reinterpret_cast<uint4*>(v + (c / 8) * kHalf + row * 128 + (c % 8) * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        return true;
      };
#pragma unroll 1
      for (int j = 0; j < n_blocks; ++j) {
        const uint32_t par = static_cast<uint32_t>(j & 1);
        const int key0 = it.k_lo + j * kBlkKeys;
        if (!__all_sync(0xffffffffu, wait_bar(&bars->s_full[t], par, abort_flag, limit_clk))) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (!live) {
          if (!clear_tail(j, key0)) break;
          mbar_arrive(&bars->p_full[t]);
          continue;
        }
        uint32_t su[4][32];
        const int valid = limit - key0;
        const bool border = __any_sync(0xffffffffu, valid < kBlkKeys);
        // The weights of the first half are computed against the reference
        // maximum as it stands, while the second half and the block's own maximum
        // are still on their way; the rare block that moves the reference (past +8
        // in base 2, so weights stay below 256) computes them again.
        float2 sum[4] = {};
        uint32_t w[32];
        auto weights = [&](int c) {  // of keys 64 c .. 64 c + 63: 32 columns of bf16 pairs
          // no key seen yet: the reference is still -inf, and every weight is 0
          const float ref = m_ref == -INFINITY ? 0.f : m_ref;
          const float2 sc2 = make_float2(scale, scale), nr2 = make_float2(-ref, -ref);
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const uint32_t* s = &su[2 * c + (i >> 4)][2 * i & 31];
            const float2 x = fma2(make_float2(__uint_as_float(s[0]), __uint_as_float(s[1])), sc2, nr2);
            const float2 e = make_float2(fast_exp2(x.x), fast_exp2(x.y));
            sum[i & 3] = add2(sum[i & 3], e);
            w[i] = pack_bf16(e.x, e.y);
          }
        };
        auto hide = [&](int c) {  // keys past this row's limit in quarter c
          if (border) {
#pragma unroll
            for (int i = 0; i < 32; ++i) su[c][i] = c * 32 + i < valid ? su[c][i] : 0xff800000u;  // -infinity
          }
        };
        float mq[8];  // eight chains
        auto raise = [&](int c) {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float x = __uint_as_float(su[c][i]);
            mq[i & 7] = c == 0 && i < 8 ? x : fmaxf(mq[i & 7], x);
          }
        };
        tmem_ld_32cols_nowait(lane_addr + t * 128, su[0]);
        tmem_ld_32cols_nowait(lane_addr + t * 128 + 32, su[1]);
        tmem_ld_wait(su[0]);
        tmem_ld_wait(su[1]);
        tmem_ld_32cols_nowait(lane_addr + t * 128 + 64, su[2]);
        tmem_ld_32cols_nowait(lane_addr + t * 128 + 96, su[3]);
        hide(0);
        hide(1);
        if (j > 0) weights(0);
        raise(0);
        raise(1);
        tmem_ld_wait(su[2]);
        tmem_ld_wait(su[3]);
        hide(2);
        hide(3);
        raise(2);
        raise(3);
        const float mx = scale * fmaxf(fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3])),
                                       fmaxf(fmaxf(mq[4], mq[5]), fmaxf(mq[6], mq[7])));
        const bool need = mx > m_ref + 8.f;
        if (j == 0 || __any_sync(0xffffffffu, need)) {
          float alpha = 1.f;
          if (need) {
            alpha = exp2f(m_ref - mx);
            m_ref = mx;
            l *= alpha;
          }
          if (j > 0) {
            // O holds every product up to block j - 1 before it is rescaled
            if (!__all_sync(0xffffffffu, wait_bar(&bars->pv_done[t], par ^ 1u, abort_flag, limit_clk))) {
              ok = false;
              break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              float o[16];
              tmem_ld_16cols(lane_addr + kTmemO + t * 128 + c * 16, o);
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] *= alpha;
              tmem_st_16cols(lane_addr + kTmemO + t * 128 + c * 16, o);
            }
          }
          sum[0] = sum[1] = sum[2] = sum[3] = make_float2(0.f, 0.f);
          weights(0);
        }
        if (!clear_tail(j, key0)) {
          ok = false;
          break;
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (c == 1) weights(1);
          tmem_st_32cols_nowait(lane_addr + t * 128 + c * 32, w);
        }
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        tc_fence_before();
        mbar_arrive(&bars->p_full[t]);
        sum[0] = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
        l += sum[0].x + sum[0].y;
      }
      // ---- clustered: the rows' part into this CTA's shared memory, once no product
      // of either tile reads it any more
      if (!PREFIX && a.clustered) {
        const bool done = ok && (!live || __all_sync(0xffffffffu, wait_bar(&bars->pv_done[t], static_cast<uint32_t>((n_blocks - 1) & 1), abort_flag, limit_clk)));
        asm volatile("bar.sync 2, %0;" ::"r"(two ? 256 : 128) : "memory");
        if (live && done) {
          tc_fence_after();
          const int pr = t * 128 + r;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t o[32];
            tmem_ld_32cols_nowait(lane_addr + kTmemO + t * 128 + c * 32, o);
            tmem_ld_wait(o);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              *reinterpret_cast<uint4*>(base + part_at(pr, 8 * c + k)) = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
          }
          *reinterpret_cast<float2*>(base + kPartStats + pr * 8) = make_float2(m_ref, l);
        }
      } else
      // ---- rows out, through this tile's Q buffer (no MMA reads it any more):
      // a warp's 32 rows as whole 256-byte lines
      if (live && ok && __all_sync(0xffffffffu, wait_bar(&bars->pv_done[t], static_cast<uint32_t>((n_blocks - 1) & 1), abort_flag, limit_clk))) {
        tc_fence_after();
        uint8_t* stage = q_tile + quarter * 8192;
        const bool final = a.dense_parts == 0;
        const float inv = 1.f / l;
        const size_t part = (PREFIX ? it.split : a.prefix_splits + it.split) * static_cast<size_t>(a.total_q) * a.hq;
        uint32_t o[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld_32cols_nowait(lane_addr + kTmemO + t * 128 + c * 32, o[c]);
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld_wait(o[c]);
        // 256 bytes of every row at a time: the row as bf16, or twice 64 of its fp32 elements
        auto copy_out = [&](int pass) {
          __syncwarp();
#pragma unroll
          for (int i0 = 0; i0 < 16; i0 += 8) {  // 16 lanes a row, eight pairs of rows in flight
            uint4 x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int row = 2 * (i0 + i) + (lane >> 4);
              x[i] = *reinterpret_cast<const uint4*>(stage + row * 256 + (((lane & 15) ^ (row & 7)) << 4));
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int row = 2 * (i0 + i) + (lane >> 4);
              const size_t dst = __shfl_sync(0xffffffffu, static_cast<unsigned long long>(out_row), row);
              if (it.row0 + t * 128 + quarter * 32 + row < it.n_rows) {
                if (final)
                  reinterpret_cast<uint4*>(a.out + dst * 128)[lane & 15] = x[i];
                else
                  reinterpret_cast<uint4*>(a.dense_o + (part + dst) * 128 + pass * 64)[lane & 15] = x[i];
              }
            }
          }
          __syncwarp();
        };
        auto put = [&](int chunk, uint4 v) {  // 16 bytes of this lane's row
          *reinterpret_cast<uint4*>(stage + lane * 256 + ((chunk ^ (lane & 7)) << 4)) = v;
        };
        if (final) {
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const uint32_t* v = &o[k >> 2][8 * k & 31];
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              w[i] = pack_bf16(__uint_as_float(v[2 * i]) * inv, __uint_as_float(v[2 * i + 1]) * inv);
            put(k, make_uint4(w[0], w[1], w[2], w[3]));
          }
          copy_out(0);
        } else {
#pragma unroll
          for (int ps = 0; ps < 2; ++ps) {
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const uint32_t* v = &o[2 * ps + (k >> 3)][4 * k & 31];
              put(k, make_uint4(v[0], v[1], v[2], v[3]));
            }
            copy_out(ps);
          }
        }
        if (row_ok) {
          if (!final)
            a.dense_st[part + out_row] = PartStat{m_ref, m_ref, l, 0.f};
          else if (a.lse != nullptr)
            a.lse[out_row] = (m_ref + log2f(l)) * 0.6931471805599453f;
        }
      }
    } else if constexpr (CODES) {  // no rows: these warps take the values off the others
      widen_blocks(base, bars, quarter, lane, 1, 2, n_blocks, it.k_hi - it.k_lo, limit_clk);
    }
  }

  if constexpr (CODES) {
    if (warp >= 12) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Cfg::kOtherRegs));
      widen_blocks(base, bars, warp & 3, lane, 0, two ? 1 : 2, n_blocks, it.k_hi - it.k_lo, limit_clk);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(bars->tmem_slot, 512);
  }
  if (threadIdx.x == 0 && *abort_flag) raise_device_error(a.c.err, QUAIL_ERR_DEVICE_TIMEOUT, 5000);
  if constexpr (!PREFIX) {
    if (a.clustered) {  // the key ranges of these rows, each in a CTA of the cluster, meet here
      __syncwarp();
      cluster_sync();
      if (softmax_warp) {
        const int parts = (tile_key_end(a, qr, it.row0) - a.seq_begin + a.seq_split - 1) / a.seq_split;
        const int rows = min(kTileRows, it.n_rows - it.row0);
        const uint32_t at = smem_u32(base);
        for (int row = it.split * 8 + warp - 4; row < rows; row += 8 * parts) {
          float2 st = make_float2(-INFINITY, 0.f);
          if (lane < parts) st = ld_cluster2(in_cta(at + kPartStats + row * 8, lane));
          float m = st.x;
#pragma unroll
          for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
          const float f = st.x == -INFINITY ? 0.f : exp2f(st.x - m);
          float sum = st.y != st.y ? st.y : f * st.y;  // a NaN sum stays one
#pragma unroll
          for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
          for (int p = 0; p < parts; ++p) {
            const float w = __shfl_sync(0xffffffffu, f, p);
            const float4 v = ld_cluster4(in_cta(at + part_at(row, lane), p));
            acc = make_float4(fmaf(v.x, w, acc.x), fmaf(v.y, w, acc.y), fmaf(v.z, w, acc.z), fmaf(v.w, w, acc.w));
          }
          const float inv = 1.f / sum;
          const int fr = it.row0 + row;
          const size_t to = static_cast<size_t>(qr.lo + fr / G) * a.hq + it.g * G + fr % G;
          *reinterpret_cast<uint2*>(a.out + to * 128 + 4 * lane) =
              make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
          if (lane == 0 && a.lse != nullptr) a.lse[to] = (m + log2f(sum)) * 0.6931471805599453f;
        }
      }
      __syncwarp();
      cluster_sync();  // no CTA leaves while another reads its part
    }
  }
  if (behind_stream) grid_dependency_wait();
}

template <bool PREFIX, bool CODES>
cudaError_t launch_tile(const SharedAttnArgs& a, const CUtensorMap& tmK, const CUtensorMap& tmV, dim3 grid,
                        int cluster, cudaStream_t st) {
  auto kern = attention_tile_kernel<PREFIX, CODES>;
  using Cfg = TileCfg<CODES>;
  static std::atomic<bool> configured[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[dev].load(std::memory_order_acquire)) {
    cudaFuncAttributes attr;
    e = cudaFuncGetAttributes(&attr, kern);
    if (e != cudaSuccess) return e;
    if (attr.numRegs != Cfg::kLaunchRegs) return cudaErrorLaunchOutOfResources;  // the register split would not add up
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(tile_smem<CODES>()));
    if (e != cudaSuccess) return e;
    configured[dev].store(true, std::memory_order_release);
  }
  count_launch();
  if (cluster == 1) return launch_pdl(kern, grid, dim3(Cfg::kThreads), tile_smem<CODES>(), st, a, tmK, tmV);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(Cfg::kThreads);
  cfg.dynamicSmemBytes = tile_smem<CODES>();
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, a, tmK, tmV);
}

}  // namespace

cudaError_t launch_attention_prefix(const SharedAttnArgs& a, const CUtensorMap& tmK, const CUtensorMap& tmV,
                                    cudaStream_t st) {
  const long rows = static_cast<long>(a.total_q) * (a.hq / a.c.hkv);
  const dim3 grid((rows + kTileRows - 1) / kTileRows, a.c.hkv, a.prefix_splits);
  return a.c.codes ? launch_tile<true, true>(a, tmK, tmV, grid, 1, st) : launch_tile<true, false>(a, tmK, tmV, grid, 1, st);
}

cudaError_t launch_attention_sequences(const SharedAttnArgs& a, const CUtensorMap& tmK, const CUtensorMap& tmV,
                                       cudaStream_t st) {
  const long rows = static_cast<long>(a.max_q) * (a.hq / a.c.hkv);
  const dim3 grid((rows + kTileRows - 1) / kTileRows * a.seq_splits, a.c.hkv, a.c.num_seqs);
  const int cluster = a.clustered ? a.seq_splits : 1;
  return a.c.codes ? launch_tile<false, true>(a, tmK, tmV, grid, cluster, st)
                   : launch_tile<false, false>(a, tmK, tmV, grid, cluster, st);
}

// Test hook: this translation unit's copy of the pipeline wait limit.
cudaError_t set_pipeline_wait_limit_cache_attention_tc(long long cycles) {
  return cudaMemcpyToSymbol(g_pipeline_wait_limit, &cycles, sizeof(cycles));
}

}  // namespace quail
