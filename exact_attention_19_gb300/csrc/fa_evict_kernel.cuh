// fa_evict_kernel.cuh -- the keys of a paged cache that gathered the least weight
// leave it, and the others move together.
//
// A sequence of len > budget + slack tokens keeps `budget` of them, for every K/V
// head its own: the first `sinks`, the last `recent`, and of those between the
// heaviest (of equal ones the lower slots).  They keep their order, so the i-th of
// them goes to slot i, which is never above its own.
//   fa_evict_select_kernel  per (sequence, K/V head): the list of kept slots, by a
//     radix selection of the smallest kept weight;
//   fa_evict_move_kernel    K, V and the weights moved by those lists; the lengths and
//     shifts.
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
  int w_vec;             // four slots of it lie on a 16-byte boundary
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
  int parts;                        // CTAs that move one head's K or V: in place those of a cluster
  unsigned int* status;
};

// An order of the bits as whole numbers: -inf < ... < -0 = 0 < ... < inf < NaN
__device__ __forceinline__ unsigned weight_order(float w) {
  if (w != w) return 0xffffffffu;
  const unsigned u = __float_as_uint(w + 0.f);  // -0 + 0 = 0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Selection: the weights of one (sequence, K/V head) are brought to shared memory
// once (in windows where they are more than fit), and the smallest kept one is found by
// its bits, 11 + 11 + 10 of them from the top: a histogram of the free weights that
// share the bits so far, and the digit at which the kept ones run out.  11 bits first
// (sign, exponent, two of the fraction), because weights share exponents: with 8 most
// counts of a warp met in the same few words.  It ends early where all weights of that
// digit stay, after two digits as a rule.  Then every warp counts what stays in its
// part of the list, and after one sum over the warps writes it, in order.
// Bound: one SM's instructions and latency per head, four weights to a thread everywhere.
// Under a profiler, caches cold: 16 heads of up to 31999 weights 35 us, 128 of up to 8192
// 15.6, 96 of up to 1024 8.4 (with one weight to a thread 55, 23 and 12).  A bracket from a
// sample of the weights before the first digit made the first 74 us of 54.
constexpr int kSelectBins = 2048;

template <int THREADS>
__global__ void __launch_bounds__(THREADS, 1) fa_evict_select_kernel(const EvictParams p) {
  constexpr int kWarps = THREADS / 32, kBinsEach = kSelectBins / THREADS;
  extern __shared__ __align__(1024) uint8_t select_smem[];
  float4* const vals = reinterpret_cast<float4*>(select_smem);  // [window / 4]
  __shared__ int hist[kSelectBins];
  __shared__ int counts[2][32];
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
  int* const kept = p.kept + static_cast<long long>(blockIdx.x) * p.most;
  const int mask = (1 << p.page_shift) - 1;
  for (int i = out + tid; i < p.most; i += THREADS) kept[i] = -1;
  if (!over) {  // stays as it is
    for (int i = tid; i < len; i += THREADS) kept[i] = i;
    if (tid == 0) p.heads[blockIdx.x] = {len, len, fork ? 0 : len, 0};
    return;
  }
  if (tid < 32) counts[0][tid] = counts[1][tid] = 0;
  if (tid == 0) first_gone = out;
  const float* const w = p.w + hk * p.w_head;
  auto load = [&](int w0) {  // the weights of tokens w0 .. of a window, four of one page to a thread
    const int n = min(p.window, len - w0);
    constexpr int kU = 4;  // in flight
    for (int j0 = 4 * tid; j0 < n; j0 += 4 * kU * THREADS) {
      int page[kU];
      float4 v[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int j = j0 + 4 * u * THREADS;
        page[u] = j < n ? coherent(table + ((w0 + j) >> p.page_shift)) : 0;
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int j = j0 + 4 * u * THREADS;
        v[u] = make_float4(0.f, 0.f, 0.f, 0.f);  // a page outside the cache: its tokens weigh nothing
        if (j >= n) continue;
        if (static_cast<unsigned>(page[u]) >= static_cast<unsigned>(p.n_pages)) {
          atomicOr(p.status, kPagedPage);
          continue;
        }
        const float* const at = w + page[u] * p.w_page + ((w0 + j) & mask);
        if (p.w_vec) {
          const uint4 x = load16(reinterpret_cast<const uint16_t*>(at));
          v[u] = make_float4(__uint_as_float(x.x), __uint_as_float(x.y), __uint_as_float(x.z), __uint_as_float(x.w));
        } else {
          v[u] = make_float4(load4(at), load4(at + 1), load4(at + 2), load4(at + 3));
        }
      }
#pragma unroll
      for (int u = 0; u < kU; ++u)
        if (j0 + 4 * u * THREADS < n) vals[j0 / 4 + u * THREADS] = v[u];
    }
  };
  const int windows = (len + p.window - 1) / p.window;
  const int lo = p.sinks, hi = len - p.recent;  // the free ones

  unsigned least = 0xffffffffu;  // the smallest order that is kept among the free ones
  int ties = 0;                  // how many of that order; below 0: all from `least` on
  bool loaded = false;
  int want = p.budget - p.sinks - p.recent;
  if (want > 0) {
    unsigned prefix = 0;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bits = pass == 2 ? 10 : 11;
      // weights that share the digits so far: order ^ prefix has none but the bits below them
      const unsigned rest = pass == 0 ? 0xffffffffu : (pass == 1 ? 0x1fffffu : 0x3ffu);
      for (int i = tid; i < kSelectBins; i += THREADS) hist[i] = 0;
      for (int k = 0; k < windows; ++k) {
        const int w0 = k * p.window, n = min(p.window, len - w0);
        if (!loaded) {
          __syncthreads();  // the window before has been read
          load(w0);
        }
        __syncthreads();
        const int f0 = lo - w0, f1 = min(hi - w0, n);
        for (int j = 4 * tid; j < n; j += 4 * THREADS) {
          const float4 v = vals[j / 4];
          const unsigned o[4] = {weight_order(v.x), weight_order(v.y), weight_order(v.z), weight_order(v.w)};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (j + e >= f0 && j + e < f1 && (o[e] ^ prefix) <= rest)
              atomicAdd(&hist[(o[e] >> shift) & ((1u << bits) - 1u)], 1);
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
      int above = __reduce_add_sync(0xffffffffu, lane < warp ? counts[0][lane] : 0) + incl - all;
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
    ties = want == found[2] ? -1 : want;
  }
  // The list: of every window each warp's part is counted, then written behind the parts before it.
  int heavier = 0, equal = 0;  // kept so far without and with the order `least`, in the windows before
  for (int k = 0; k < windows; ++k) {
    const int w0 = k * p.window, n = min(p.window, len - w0);
    if (!loaded) {
      __syncthreads();
      load(w0);
    }
    __syncthreads();
    const int part = ((n + kWarps - 1) / kWarps + 127) & ~127;  // of a warp
    const int j0 = min(n, warp * part), j1 = min(n, j0 + part);
    const int f0 = lo - w0, f1 = hi - w0;
    // which of tokens j .. j + 3 stay for sure, and which if the ties go that far
    auto stays = [&](int j, unsigned& sure, unsigned& tie) {
      const float4 v = j < j1 ? vals[j / 4] : make_float4(0.f, 0.f, 0.f, 0.f);
      const unsigned o[4] = {weight_order(v.x), weight_order(v.y), weight_order(v.z), weight_order(v.w)};
      sure = tie = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool held = j + e < f0 || j + e >= f1;
        const bool in = j + e < j1;
        sure |= (in && (held || o[e] > least || (ties < 0 && o[e] == least))) ? 1u << e : 0u;
        tie |= (in && !held && ties > 0 && o[e] == least) ? 1u << e : 0u;
      }
    };
    int a = 0, t = 0;
    for (int j = j0 + 4 * lane; j < j0 + part; j += 128) {
      unsigned sure, tie;
      stays(j, sure, tie);
      a += __popc(sure);
      t += __popc(tie);
    }
    a = __reduce_add_sync(0xffffffffu, a);
    t = __reduce_add_sync(0xffffffffu, t);
    if (lane == 0) {
      counts[0][warp] = a;
      counts[1][warp] = t;
    }
    __syncthreads();
    a = counts[0][lane];
    t = counts[1][lane];
    const int all_a = __reduce_add_sync(0xffffffffu, a), all_t = __reduce_add_sync(0xffffffffu, t);
    a = heavier + __reduce_add_sync(0xffffffffu, lane < warp ? a : 0);
    t = equal + __reduce_add_sync(0xffffffffu, lane < warp ? t : 0);
    heavier += all_a;
    equal += all_t;
    int gone = 0x7fffffff;
    for (int j = j0 + 4 * lane; j - 4 * lane < j1; j += 128) {
      unsigned sure, tie;
      stays(j, sure, tie);
      // kept ones in the lanes before: sums of both kinds in one word
      const int mine = __popc(sure) | __popc(tie) << 16;
      int incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
      }
      const int all = __shfl_sync(0xffffffffu, incl, 31);
      int at = a + ((incl - mine) & 0xffff), before = t + ((incl - mine) >> 16);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool is_sure = (sure >> e) & 1u, is_tie = (tie >> e) & 1u;
        if (is_sure || (is_tie && before < ties)) kept[at + min(before, max(ties, 0))] = w0 + j + e;
        else if (j + e < j1) gone = min(gone, w0 + j + e);
        at += is_sure;
        before += is_tie;
      }
      a += all & 0xffff;
      t += all >> 16;
    }
    gone = __reduce_min_sync(0xffffffffu, gone);
    if (lane == 0) atomicMin(&first_gone, gone);  // where the first one goes, the list leaves its slots
    loaded = false;
  }
  __syncthreads();
  if (tid == 0) p.heads[blockIdx.x] = {len, out, fork ? 0 : first_gone, 0};
}

// The rows of K or V, or the weights, of one (sequence, K/V head), by one cluster (by any
// CTAs where they go to other pages).  A round takes
// kRows * kU rows of each CTA; all of a round are read before any is written, and as a
// destination lies at or below its own source, it lies below the sources of later
// rounds, so that one barrier of the cluster stands between a round's loads and its
// stores and nothing after them.  Into other pages no barrier is needed.
// Bound: memory; a round in place waits for its loads (a cluster has its rows of the
// next round looked up meanwhile), which shows where few rows are moved: 128 heads of up to
// 8192 halved, K and V of 128, 74 us cold, 16 heads of up to 31999 to 8000 into other pages 32.
constexpr int kMoveThreads = 512;

template <int D>
__global__ void __launch_bounds__(kMoveThreads, 2) fa_evict_move_kernel(const EvictParams p) {
  constexpr int kLanes = D / 8;  // 16 bytes each
  constexpr int kU = 8;          // in flight per thread
  constexpr int kRows = kMoveThreads / kLanes;
  grid_wait();
  grid_release();
  const int ranks = p.parts, rank = blockIdx.x % ranks;
  const int unit = blockIdx.x / ranks, kv = unit % 3, bh = unit / 3, b = bh / p.Hk, hk = bh % p.Hk;  // 2: the weights
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
  auto page_of = [&](const int* pages, int slot) -> int {  // -1: outside the cache
    const int page = coherent(pages + (slot >> p.page_shift));
    if (static_cast<unsigned>(page) < static_cast<unsigned>(p.n_pages)) return page;
    atomicOr(p.status, kPagedPage);
    return -1;
  };
  // between a round's loads and its stores
  auto all_read = [&]() {
    if (fork) return;
    __syncwarp();
    if (ranks > 1) cluster_sync();
    else __syncthreads();
  };
  if (kv == 2) {
    float* const w = p.w + hk * p.w_head;
    for (int i0 = h.first; i0 < h.out; i0 += kMoveThreads * kU * ranks) {
      float v[kU];
      unsigned there = 0;
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int i = i0 + (rank * kU + u) * kMoveThreads + static_cast<int>(threadIdx.x);
        if (i >= h.out) continue;
        const int slot = coherent(kept + i), page = page_of(table, slot);
        if (page < 0) continue;
        there |= 1u << u;
        v[u] = load4(w + page * p.w_page + (slot & mask));
      }
      all_read();
#pragma unroll
      for (int u = 0; u < kU; ++u)
        if ((there >> u) & 1u) {
          const int i = i0 + (rank * kU + u) * kMoveThreads + static_cast<int>(threadIdx.x), page = page_of(to, i);
          if (page >= 0) w[page * p.w_page + (i & mask)] = v[u];
        }
    }
    return;
  }
  uint16_t* const cache = p.cache[kv] + hk * p.head[kv] + threadIdx.x % kLanes * 8;
  auto place = [&](const int* pages, int slot) -> uint16_t* {
    const int page = page_of(pages, slot);
    return page < 0 ? nullptr : cache + page * p.page[kv] + (slot & mask) * p.token[kv];
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
    all_read();
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if ((there >> u) & 1u) {
        uint16_t* const at = place(to, i0 + row + u * kRows);
        if (at) *reinterpret_cast<uint4*>(at) = v[u];
      }
  }
}

}  // namespace fa
