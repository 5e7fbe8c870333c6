// Page tables that follow the sequences' lengths. The pool's free pages are a ring: a
// growing sequence takes from its head, a shrinking one appends to its end, so that in
// one call what is given back is never what is taken, and no block waits for another.
// With own(n) = max(n, prefix) and P(n) = own(n) / 16, rounded up, sequence b lacks
// P(new) - P(old) pages and gets own(new) - own(old) tokens; growing sequences are granted
// in order while the running sums of both fit. The sums never fall, so the granted ones
// are those up to the first that does not fit, and their own running sums are the same.
//
// Bound by latency: every block sums up all sequences for itself (8 bytes each, from L2)
// instead of waiting for one that does, then takes its share of the sequences (a warp
// each: pages, lengths) and of the tokens (four a thread, by search).
#include <algorithm>
#include <type_traits>

#include "launch.cuh"
#include "quail_internal.h"
#include "sm103.cuh"
#include "tree.h"

namespace quail {

namespace {

constexpr int kPage = 16;

struct Want {
  int first, last;  // own(old), own(new)
  int take, give;   // pages
  int tokens;
  bool ok;          // both lengths valid
  bool grows;
};
__device__ __forceinline__ Want want(const ResizeArgs& a, int b) {
  Want w{};
  const int o = a.old_len[b], n = a.new_len[b];
  const long long cap = static_cast<long long>(a.c.max_pages) * kPage;
  w.ok = o >= 0 && n >= 0 && o <= cap && n <= cap && (o == 0 || o >= a.prefix_len) && (n == 0 || n >= a.prefix_len);
  if (!w.ok) return w;
  w.grows = n > o;
  w.first = max(o, a.prefix_len);
  w.last = max(n, a.prefix_len);
  // (x - 1) / 16 + 1 would be 1 for 0; lengths reach 2^31 - 16, so no sum with 15
  const int pf = w.first / kPage + (w.first % kPage != 0), pl = w.last / kPage + (w.last % kPage != 0);
  if (w.grows) {
    w.take = pl - pf;
    w.tokens = w.last - w.first;
  } else {
    w.give = pf - pl;
  }
  return w;
}

struct Sums {
  long long take, tokens, give;
};
__device__ __forceinline__ Sums operator+(const Sums& x, const Sums& y) {
  return {x.take + y.take, x.tokens + y.tokens, x.give + y.give};
}
__device__ __forceinline__ Sums shfl_up(const Sums& x, int d) {
  return {__shfl_up_sync(0xffffffffu, x.take, d), __shfl_up_sync(0xffffffffu, x.tokens, d),
          __shfl_up_sync(0xffffffffu, x.give, d)};
}
__device__ __forceinline__ Sums warp_scan(Sums x, int lane) {  // inclusive
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const Sums y = shfl_up(x, d);
    if (lane >= d) x = x + y;
  }
  return x;
}

template <int THREADS>
__global__ void __launch_bounds__(THREADS) cache_resize_kernel(ResizeArgs a) {
  constexpr int kWarps = THREADS / 32;
  __shared__ Sums s_scan[THREADS + 1];  // before the run of thread i
  __shared__ Sums s_warp[kWarps];
  __shared__ long long s_take[kWarps], s_tokens[kWarps];
  grid_dependency_wait();
  const int B = a.c.num_seqs, N = a.c.num_pages, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int per = (B + THREADS - 1) / THREADS;
  const int b0 = min(B, static_cast<int>(threadIdx.x) * per), b1 = min(B, b0 + per);
  int head = a.state[0], count = a.state[1];
  const bool state_ok = head >= 0 && head < N && count >= 0 && count <= N;
  if (!state_ok) head = count = 0;
  Sums mine{0, 0, 0};
  for (int b = b0; b < b1; ++b) {
    const Want w = want(a, b);
    if (!w.ok && blockIdx.x == 0) raise_device_error(a.c.err, QUAIL_ERR_DEVICE_BOUNDS, b);
    mine = mine + Sums{w.take, w.tokens, w.give};
  }
  const Sums in_warp = warp_scan(mine, lane);
  if (lane == 31) s_warp[warp] = in_warp;
  __syncthreads();
  Sums before{0, 0, 0};
  for (int i = 0; i < warp; ++i) before = before + s_warp[i];
  s_scan[threadIdx.x + 1] = before + in_warp;
  if (threadIdx.x == 0) s_scan[0] = Sums{0, 0, 0};
  // the running sums at the last granted sequence
  const long long room = a.token_seq != nullptr ? a.max_tokens : 0x7fffffffffffLL;
  long long take = 0, tokens = 0;
  {
    Sums at = before + in_warp;
    at = Sums{at.take - mine.take, at.tokens - mine.tokens, 0};
    for (int b = b0; b < b1; ++b) {
      const Want w = want(a, b);
      at = at + Sums{w.take, w.tokens, 0};
      if (w.grows && at.take <= count && at.tokens <= room) {
        take = at.take;
        tokens = at.tokens;
      }
    }
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    take = max(take, __shfl_xor_sync(0xffffffffu, take, d));
    tokens = max(tokens, __shfl_xor_sync(0xffffffffu, tokens, d));
  }
  if (lane == 0) {
    s_take[warp] = take;
    s_tokens[warp] = tokens;
  }
  __syncthreads();
  for (int i = 0; i < kWarps; ++i) {
    take = max(take, s_take[i]);
    tokens = max(tokens, s_tokens[i]);
  }
  const long long give = s_scan[THREADS].give;
  // a ring that is no ring, or more pages back than it can hold: nothing shrinks
  const bool give_ok = state_ok && count + give <= N;
  if (!give_ok && blockIdx.x == 0 && threadIdx.x == 0) raise_device_error(a.c.err, QUAIL_ERR_DEVICE_BOUNDS, -1);
  const int pp = a.prefix_len / kPage;

  // ---- sequences, a warp each: table, ring, granted length, first token
  for (int b = blockIdx.x * kWarps + warp; b < B; b += gridDim.x * kWarps) {
    const int run = b / per, r0 = run * per;
    Sums at{0, 0, 0};
    for (int i = r0 + lane; i < b; i += 32) {
      const Want w = want(a, i);
      at = at + Sums{w.take, w.tokens, w.give};
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
      at = at + Sums{__shfl_xor_sync(0xffffffffu, at.take, d), __shfl_xor_sync(0xffffffffu, at.tokens, d),
                     __shfl_xor_sync(0xffffffffu, at.give, d)};
    at = at + s_scan[run];
    const Want w = want(a, b);
    const int old = a.old_len[b];
    const bool granted = w.ok && (w.grows ? at.take + w.take <= count && at.tokens + w.tokens <= room : give_ok);
    if (lane == 0) {
      a.granted[b] = granted ? a.new_len[b] : old;
      a.offsets[b] = static_cast<int>(min(at.tokens, tokens));
    }
    if (!granted) continue;
    int* row = a.table + static_cast<size_t>(b) * a.c.max_pages;
    const int pf = w.first / kPage + (w.first % kPage != 0);
    if (w.grows) {
      if (old == 0)
        for (int p = lane; p < pp; p += 32) row[p] = a.prefix_pages[p];
      for (int p = lane; p < w.take; p += 32) {
        long long i = head + at.take + p;
        if (i >= N) i -= N;
        row[pf + p] = a.ring[i];
      }
    } else {
      const int pl = pf - w.give;
      for (int p = lane; p < w.give; p += 32) {
        long long i = static_cast<long long>(head) + count + at.give + p;
        i -= i >= N ? N : 0;
        a.ring[i >= N ? i - N : i] = row[pl + p];
        row[pl + p] = -1;
      }
    }
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) a.offsets[B] = static_cast<int>(tokens);

  // ---- tokens, four a thread
  if (a.token_seq != nullptr) {
    for (long long t0 = 4LL * (blockIdx.x * THREADS + threadIdx.x); t0 < a.max_tokens; t0 += 4LL * gridDim.x * THREADS) {
      int seq[4], pos[4];
      int b = -1;
      long long start = 0, end = 0;  // tokens of sequence b
      int first = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const long long t = t0 + k;
        seq[k] = -1;
        pos[k] = 0;
        if (t >= tokens) continue;
        if (b < 0) {
          int lo = 0, hi = THREADS;  // s_scan[lo].tokens <= t < s_scan[hi].tokens
          while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (s_scan[mid].tokens <= t)
              lo = mid;
            else
              hi = mid;
          }
          b = lo * per - 1;
          end = s_scan[lo].tokens;
        }
        while (t >= end && b + 1 < B) {
          const Want w = want(a, ++b);
          start = end;
          end += w.tokens;
          first = w.first;
        }
        seq[k] = b;
        pos[k] = first + static_cast<int>(t - start);
      }
      if (t0 + 4 <= a.max_tokens) {
        *reinterpret_cast<int4*>(a.token_seq + t0) = make_int4(seq[0], seq[1], seq[2], seq[3]);
        *reinterpret_cast<int4*>(a.token_pos + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (t0 + k < a.max_tokens) {
            a.token_seq[t0 + k] = seq[k];
            a.token_pos[t0 + k] = pos[k];
          }
      }
    }
  }

  // ---- the ring's new state, by the last block: all have read the old one
  __syncthreads();
  if (threadIdx.x == 0 && state_ok) {
    bool last = gridDim.x == 1;
    if (!last) {
      __threadfence();
      last = atomicAdd(a.state + 2, 1) == static_cast<int>(gridDim.x) - 1;
    }
    if (last) {
      a.state[0] = static_cast<int>((head + take) % N);
      a.state[1] = static_cast<int>(count - take + (give_ok ? give : 0));
      a.state[2] = 0;
    }
  }
}

}  // namespace

cudaError_t launch_cache_resize(const ResizeArgs& a, int num_sms, cudaStream_t st) {
  count_launch();
  const auto launch = [&](auto threads) {
    constexpr int kThreads = decltype(threads)::value;
    const long long by_tokens = a.token_seq != nullptr ? (a.max_tokens + 4LL * kThreads - 1) / (4LL * kThreads) : 0;
    const long long by_seqs = (a.c.num_seqs + kThreads / 32 - 1) / (kThreads / 32);
    const int grid = static_cast<int>(std::max(1LL, std::min<long long>(num_sms, std::max(by_tokens, by_seqs))));
    return launch_pdl(cache_resize_kernel<kThreads>, dim3(grid), dim3(kThreads), 0, st, a);
  };
  // Few sequences: eight warps, whose sums take a fourth of the time to add up. 4 sequences
  // 7.4 us with 1,024 threads, 4.0 with 256; 512 that gain 260,000 tokens 10.4 and 6.4.
  if (a.c.num_seqs <= 1024) return launch(std::integral_constant<int, 256>{});
  return launch(std::integral_constant<int, 1024>{});
}

}  // namespace quail
