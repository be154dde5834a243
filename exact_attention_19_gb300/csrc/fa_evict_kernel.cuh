// fa_evict_kernel.cuh -- the keys of a paged cache that gathered the least weight
// leave it, and the others move together.
//
// A sequence of len > budget + slack tokens keeps `budget` of them, for every K/V
// head its own: the first `sinks`, the last `recent`, and of those between the
// heaviest (of equal ones the lower slots).  They keep their order, so the i-th of
// them goes to slot i, which is never above its own.
//   fa_evict_select_kernel  per (sequence, K/V head): the list of kept slots, by a
//     radix selection of the smallest kept weight, and the weights moved;
//   fa_evict_move_kernel    K and V moved by those lists; the lengths and shifts.
#pragma once

#include "fa_cache_ptx.cuh"
#include "fa_paged_kernel.cuh"

namespace fa {

struct EvictHead {  // what the selection leaves for the move, per (sequence, K/V head)
  int len, out;     // tokens before and after
  int first;        // first place in the list whose token has to move
  int unused;
};

struct EvictParams {
  uint16_t* cache[2];  // K, V
  long long page[2], head[2], token[2];
  float* w;            // [n_pages, Hk, page]
  long long w_page, w_head;
  const int* table;      // [B, max_pages]
  const int* table_out;  // [B, out_pages], or the same as table
  const int* lens;
  int* lens_out;         // may be lens
  int* shift;            // or nullptr
  int* kept;             // [B, Hk, most]
  EvictHead* heads;      // workspace
  int B, Hk, n_pages, max_pages, out_pages, page_shift, capacity;
  int budget, recent, sinks, most;  // most = budget + slack
  int window;                       // weights that the selection holds in shared memory
  unsigned int* status;
};

// An order of the bits as whole numbers: -inf < ... < -0 = 0 < ... < inf < NaN
__device__ __forceinline__ unsigned weight_order(float w) {
  if (w != w) return 0xffffffffu;
  const unsigned u = __float_as_uint(w + 0.f);  // -0 + 0 = 0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Selection: the weights of one (sequence, K/V head) are brought to shared memory
// once (in windows where they are more than fit, the last window staying), and the
// smallest kept one is found by its bits, 11 + 11 + 10 of them from the top: a
// histogram of the free weights that share the bits so far, and the digit at which the
// kept ones run out.  11 bits first (sign, exponent, two of the fraction), because
// weights share exponents: with 8 most counts of a warp met in the same few words.
// It ends early where all weights of that digit stay, after two digits as a rule.
// Then every warp counts what stays in its part of the list, and after one sum over
// the warps writes it, in order.
// Bound: latency (lengths, pages, weights, then a few barriers to a digit).
constexpr int kSelectBins = 2048;

template <int THREADS>
__global__ void __launch_bounds__(THREADS, 1) fa_evict_select_kernel(const EvictParams p) {
  constexpr int kWarps = THREADS / 32, kBinsEach = kSelectBins / THREADS;
  extern __shared__ float vals[];  // [window]
  __shared__ int hist[kSelectBins];
  __shared__ int counts[2][kWarps];
  __shared__ int found[3];  // digit, how many of its weights stay, how many there are
  __shared__ int first_gone;
  grid_wait();
  grid_release();
  const int b = blockIdx.x / p.Hk, hk = blockIdx.x % p.Hk;
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  const int raw = coherent(p.lens + b);
  const int len = max(0, min(raw, p.capacity));
  if (raw > p.capacity && tid == 0) atomicOr(p.status, kPagedPage);
  const bool fork = p.table_out != p.table, over = len > p.most;
  const int out = over ? p.budget : len;
  const int* const table = p.table + static_cast<long long>(b) * p.max_pages;
  const int* const to = p.table_out + static_cast<long long>(b) * p.out_pages;
  int* const kept = p.kept + static_cast<long long>(blockIdx.x) * p.most;
  const int mask = (1 << p.page_shift) - 1;
  for (int i = out + tid; i < p.most; i += THREADS) kept[i] = -1;
  if (!over && !fork) {  // stays as it is
    for (int i = tid; i < len; i += THREADS) kept[i] = i;
    if (tid == 0) p.heads[blockIdx.x] = {len, len, len, 0};
    return;
  }
  float* const w = p.w + hk * p.w_head;
  auto load = [&](int w0) {  // the weights of tokens w0 .. of a window
    const int n = min(p.window, len - w0);
    constexpr int kU = 8;  // in flight
    for (int j0 = tid; j0 < n; j0 += kU * THREADS) {
      int page[kU];
      float v[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u)
        page[u] = j0 + u * THREADS < n ? coherent(table + ((w0 + j0 + u * THREADS) >> p.page_shift)) : 0;
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int j = j0 + u * THREADS;
        v[u] = 0.f;  // a page outside the cache: its tokens weigh nothing
        if (j < n) {
          if (static_cast<unsigned>(page[u]) < static_cast<unsigned>(p.n_pages)) v[u] = load4(w + page[u] * p.w_page + ((w0 + j) & mask));
          else atomicOr(p.status, kPagedPage);
        }
      }
#pragma unroll
      for (int u = 0; u < kU; ++u)
        if (j0 + u * THREADS < n) vals[j0 + u * THREADS] = v[u];
    }
  };
  const int windows = (len + p.window - 1) / p.window;
  const int lo = p.sinks, hi = len - p.recent;  // the free ones

  unsigned least = 0;  // the smallest order that is kept among the free ones
  int ties = 0;        // how many of that order
  bool loaded = false, from_least = false;
  if (over) {
    int want = p.budget - p.sinks - p.recent;
    if (want == 0) {
      least = 0xffffffffu;
    } else {
      unsigned prefix = 0;
#pragma unroll 1
      for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bits = pass == 2 ? 10 : 11, above_bits = shift + bits;
        for (int i = tid; i < kSelectBins; i += THREADS) hist[i] = 0;
        for (int k = 0; k < windows; ++k) {
          const int w0 = k * p.window;
          if (!loaded) {
            __syncthreads();  // the window before has been read
            load(w0);
          }
          __syncthreads();
          const int j1 = min(hi - w0, min(p.window, len - w0));
          for (int j = max(lo - w0, 0) + tid; j < j1; j += THREADS) {
            const unsigned o = weight_order(vals[j]);
            if (pass == 0 || (o >> above_bits) == (prefix >> above_bits))
              atomicAdd(&hist[(o >> shift) & ((1u << bits) - 1u)], 1);
          }
        }
        loaded = windows == 1;
        __syncthreads();
        // thread t holds the bins kSelectBins - 1 - kBinsEach t downwards, so sums run from the heaviest
        int n[kBinsEach], all = 0;
#pragma unroll
        for (int i = 0; i < kBinsEach; ++i) {
          n[i] = hist[kSelectBins - 1 - kBinsEach * tid - i];
          all += n[i];
        }
        int incl = all;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int up = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += up;
        }
        if (lane == 31) counts[0][warp] = incl;
        __syncthreads();
        int above = incl - all;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) above += i < warp ? counts[0][i] : 0;
        if (above < want && want <= above + all) {
#pragma unroll
          for (int i = 0; i < kBinsEach; ++i) {
            if (above < want && want <= above + n[i]) {
              found[0] = kSelectBins - 1 - kBinsEach * tid - i;
              found[1] = want - above;
              found[2] = n[i];
            }
            above += n[i];
          }
        }
        __syncthreads();
        prefix |= static_cast<unsigned>(found[0]) << shift;
        want = found[1];
        if (want == found[2]) break;
      }
      least = prefix;  // zeros below the digits that were looked at
      ties = want;     // those with these digits; all of them where that ended the search, so their order from `least` on
      from_least = want == found[2];
    }
  }
  // the list.  All of a window's weights have been read before any moves, and those that do land at or below their own
  // slots, so below the windows to come.
  if (tid == 0) first_gone = fork ? 0 : out;
  int heavier = 0, equal = 0;  // kept so far without and with the order `least`, in the windows before
  for (int k = 0; k < windows; ++k) {
    const int w0 = k * p.window, n = min(p.window, len - w0);
    if (!loaded) {
      __syncthreads();
      load(w0);
    }
    __syncthreads();
    const int part = ((n + kWarps - 1) / kWarps + 31) & ~31;  // of a warp
    const int j0 = min(n, warp * part), j1 = min(n, j0 + part);
    auto stays = [&](int j, bool& sure, bool& tie) {
      sure = tie = false;
      if (j >= j1) return;
      const int slot = w0 + j;
      if (!over || slot < lo || slot >= hi) {
        sure = true;
      } else {
        const unsigned o = weight_order(vals[j]);
        sure = from_least ? o >= least : o > least;
        tie = !from_least && ties > 0 && o == least;
      }
    };
    int a = 0, t = 0;
#pragma unroll 4
    for (int j = j0; j < j1; j += 32) {
      bool sure, tie;
      stays(j + lane, sure, tie);
      a += __popc(__ballot_sync(0xffffffffu, sure));
      t += __popc(__ballot_sync(0xffffffffu, tie));
    }
    if (lane == 0) {
      counts[0][warp] = a;
      counts[1][warp] = t;
    }
    __syncthreads();
    a = heavier;
    t = equal;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      a += i < warp ? counts[0][i] : 0;
      t += i < warp ? counts[1][i] : 0;
      heavier += counts[0][i];
      equal += counts[1][i];
    }
    int gone = 0x7fffffff;
#pragma unroll 4
    for (int j = j0; j < j1; j += 32) {
      bool sure, tie;
      stays(j + lane, sure, tie);
      const unsigned sure_bits = __ballot_sync(0xffffffffu, sure), tie_bits = __ballot_sync(0xffffffffu, tie);
      const unsigned below = (1u << lane) - 1u;
      const int before = t + __popc(tie_bits & below), slot = w0 + j + lane;
      if (sure || (tie && before < ties)) {
        const int i = a + __popc(sure_bits & below) + min(before, ties);
        kept[i] = slot;
        if (fork || i != slot) {
          const int page = coherent(to + (i >> p.page_shift));
          if (static_cast<unsigned>(page) < static_cast<unsigned>(p.n_pages)) w[page * p.w_page + (i & mask)] = vals[j + lane];
          else atomicOr(p.status, kPagedPage);
        }
      } else if (j + lane < j1) {
        gone = min(gone, slot);
      }
      a += __popc(sure_bits);
      t += __popc(tie_bits);
    }
    gone = __reduce_min_sync(0xffffffffu, gone);
    if (lane == 0) atomicMin(&first_gone, gone);  // where the first one goes, the list leaves its slots
    loaded = false;
  }
  __syncthreads();
  if (tid == 0) p.heads[blockIdx.x] = {len, out, first_gone, 0};
}

// The rows of K or V of one (sequence, K/V head), by one cluster.  A round takes
// kRows * kU rows of each CTA; all of a round are read before any is written, and as a
// destination lies at or below its own source, it lies below the sources of later
// rounds, so that one barrier of the cluster stands between a round's loads and its
// stores and nothing after them.  Into other pages no barrier is needed.
constexpr int kMoveThreads = 512;

template <int D>
__global__ void __launch_bounds__(kMoveThreads, 2) fa_evict_move_kernel(const EvictParams p) {
  constexpr int kLanes = D / 8;  // 16 bytes each
  constexpr int kU = 8;          // in flight per thread
  constexpr int kRows = kMoveThreads / kLanes;
  grid_wait();
  grid_release();
  const int ranks = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
  const int unit = blockIdx.x / ranks, kv = unit & 1, bh = unit >> 1, b = bh / p.Hk, hk = bh % p.Hk;
  const EvictHead h = p.heads[bh];
  if (threadIdx.x == 0 && kv == 0 && hk == 0 && rank == 0) {
    p.lens_out[b] = h.out;
    if (p.shift) p.shift[b] += h.len - h.out;
  }
  const bool fork = p.table_out != p.table;
  const int* const kept = p.kept + static_cast<long long>(bh) * p.most;
  const int* const table = p.table + static_cast<long long>(b) * p.max_pages;
  const int* const to = p.table_out + static_cast<long long>(b) * p.out_pages;
  const int mask = (1 << p.page_shift) - 1;
  uint16_t* const cache = p.cache[kv] + hk * p.head[kv] + threadIdx.x % kLanes * 8;
  auto place = [&](const int* pages, int slot) -> uint16_t* {
    const int page = coherent(pages + (slot >> p.page_shift));
    if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.n_pages)) {
      atomicOr(p.status, kPagedPage);
      return nullptr;
    }
    return cache + page * p.page[kv] + (slot & mask) * p.token[kv];
  };
  const int step = kRows * kU, row = rank * step + static_cast<int>(threadIdx.x) / kLanes;
  const uint16_t* from[kU];  // of the round to come
  auto look = [&](int i0) {
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int i = i0 + row + u * kRows;
      from[u] = i < h.out ? place(table, coherent(kept + i)) : nullptr;
    }
  };
  look(h.first);
  for (int i0 = h.first; i0 < h.out; i0 += step * ranks) {
    uint4 v[kU];
    unsigned there = 0;
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if (from[u]) {
        there |= 1u << u;
        v[u] = load16(from[u]);
      }
    look(i0 + step * ranks);
    if (!fork) {
      __syncwarp();
      if (ranks > 1) cluster_sync();
      else __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if ((there >> u) & 1u) {
        uint16_t* const at = place(to, i0 + row + u * kRows);
        if (at) *reinterpret_cast<uint4*>(at) = v[u];
      }
  }
}

}  // namespace fa
