// fa_evict_kernel.cuh -- the keys of a paged cache that gathered the least weight
// leave it, and the others move together.
//
// A sequence of len > budget + slack tokens keeps `budget` of them, for every K/V
// head its own: the first `sinks`, the last `recent`, and of those between the
// heaviest (of equal ones the lower slots).  They keep their order, so the i-th of
// them goes to slot i, which is never above its own.
//   fa_evict_select_kernel  per (sequence, K/V head): the list of kept slots, by a
//     radix selection of the smallest kept weight, and the weights moved;
//   fa_evict_move_kernel    K and V moved by those lists, the lengths.
#pragma once

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
  unsigned int* status;
};

// An order of the bits as whole numbers: -inf < ... < -0 = 0 < ... < inf < NaN
__device__ __forceinline__ unsigned weight_order(float w) {
  if (w != w) return 0xffffffffu;
  const unsigned u = __float_as_uint(w + 0.f);  // -0 + 0 = 0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

constexpr int kSelectThreads = 1024;

__global__ void __launch_bounds__(kSelectThreads, 1) fa_evict_select_kernel(const EvictParams p) {
  constexpr int kWarps = kSelectThreads / 32;
  __shared__ int hist[256];
  __shared__ unsigned found[2];  // digit, how many of the digit's keys are kept
  __shared__ int counts[2][kWarps];
  __shared__ int first_gone;
  grid_wait();
  grid_release();
  const int b = blockIdx.x / p.Hk, hk = blockIdx.x % p.Hk;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int raw = coherent(p.lens + b);
  const int len = max(0, min(raw, p.capacity));
  if (raw > p.capacity && threadIdx.x == 0) atomicOr(p.status, kPagedPage);
  const bool fork = p.table_out != p.table, over = len > p.most;
  const int* const table = p.table + static_cast<long long>(b) * p.max_pages;
  const int* const to = p.table_out + static_cast<long long>(b) * p.out_pages;
  int* const kept = p.kept + static_cast<long long>(blockIdx.x) * p.most;
  const int mask = (1 << p.page_shift) - 1;
  auto weight_at = [&](int j) -> float* {
    const int page = coherent(table + (j >> p.page_shift));
    if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.n_pages)) {
      atomicOr(p.status, kPagedPage);
      return nullptr;
    }
    return p.w + page * p.w_page + hk * p.w_head + (j & mask);
  };
  auto put_weight = [&](int i, float v) {
    const int page = coherent(to + (i >> p.page_shift));
    if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.n_pages)) atomicOr(p.status, kPagedPage);
    else p.w[page * p.w_page + hk * p.w_head + (i & mask)] = v;
  };
  auto order_at = [&](int j) -> unsigned {
    const float* const w = weight_at(j);
    return weight_order(w ? *w : 0.f);
  };
  const int out = over ? p.budget : len;
  if (threadIdx.x == 0) first_gone = fork ? 0 : out;

  unsigned least = 0;  // the smallest order that is kept among the free ones
  int ties = 0;        // how many of that order
  const int lo = p.sinks, hi = len - p.recent;  // the free ones
  if (over) {
    int want = p.budget - p.sinks - p.recent;
    if (want == 0) {
      least = 0xffffffffu;
    } else {
      unsigned prefix = 0;
      for (int shift = 24; shift >= 0; shift -= 8) {
        if (threadIdx.x < 256) hist[threadIdx.x] = 0;
        __syncthreads();
        for (int j = lo + static_cast<int>(threadIdx.x); j < hi; j += kSelectThreads) {
          const unsigned o = order_at(j);
          if (shift == 24 || (o >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(o >> shift) & 255u], 1);
        }
        __syncthreads();
        if (warp == 0) {  // lane l holds digits 255 - 8 l .. 248 - 8 l, from the heaviest down
          int n[8], all = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            n[i] = hist[255 - 8 * lane - i];
            all += n[i];
          }
          int incl = all;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += up;
          }
          int above = incl - all;
          if (above < want && want <= incl) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              if (above < want && want <= above + n[i]) {
                found[0] = 255 - 8 * lane - i;
                found[1] = want - above;
              }
              above += n[i];
            }
          }
        }
        __syncthreads();
        prefix |= found[0] << shift;
        want = static_cast<int>(found[1]);
      }
      least = prefix;
      ties = want;
    }
  }
  // the list, in chunks of one slot per thread; a chunk's weights are read before any of them moves, and its
  // destinations lie at or below its own slots
  int heavier = 0, equal = 0;  // kept so far without and with the order `least`, over the chunks before
  for (int j0 = 0; j0 < len; j0 += kSelectThreads) {
    const int j = j0 + static_cast<int>(threadIdx.x);
    float v = 0.f;
    bool sure = false, tie = false;
    if (j < len && (over || fork)) {
      const float* const w = weight_at(j);
      if (w) v = *w;
    }
    if (j < len) {
      if (!over || j < lo || j >= hi) {
        sure = true;
      } else {
        const unsigned o = weight_order(v);
        sure = o > least;
        tie = ties > 0 && o == least;
      }
    }
    const unsigned sure_bits = __ballot_sync(0xffffffffu, sure), tie_bits = __ballot_sync(0xffffffffu, tie);
    if (lane == 0) {
      counts[0][warp] = __popc(sure_bits);
      counts[1][warp] = __popc(tie_bits);
    }
    __syncthreads();
    int a = heavier, t = equal;
    for (int i = 0; i < kWarps; ++i) {
      if (i < warp) {
        a += counts[0][i];
        t += counts[1][i];
      }
      heavier += counts[0][i];
      equal += counts[1][i];
    }
    const unsigned below = (1u << lane) - 1u;
    a += __popc(sure_bits & below);
    t += __popc(tie_bits & below);
    if (sure || (tie && t < ties)) {
      const int i = a + min(t, ties);
      kept[i] = j;
      if ((over || fork) && (fork || i != j)) put_weight(i, v);
    } else if (j < len) {
      atomicMin(&first_gone, j);  // where the first one goes, the list leaves its slots
    }
    __syncthreads();
  }
  for (int i = out + static_cast<int>(threadIdx.x); i < p.most; i += kSelectThreads) kept[i] = -1;
  if (threadIdx.x == 0) p.heads[blockIdx.x] = {len, out, first_gone, 0};
}

constexpr int kMoveThreads = 512;

template <int D>
__global__ void __launch_bounds__(kMoveThreads) fa_evict_move_kernel(const EvictParams p) {
  constexpr int kLanes = D / 8;  // 16 bytes each
  constexpr int kU = 8;          // in flight per thread
  constexpr int kRows = kMoveThreads / kLanes;
  grid_wait();
  grid_release();
  const int kv = blockIdx.x & 1, bh = blockIdx.x >> 1, b = bh / p.Hk, hk = bh % p.Hk;
  const EvictHead h = p.heads[bh];
  if (threadIdx.x == 0 && kv == 0 && hk == 0) {
    p.lens_out[b] = h.out;
    if (p.shift) p.shift[b] += h.len - h.out;
  }
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
  // rows of a round are all read before any is written: a destination lies at or below its own source, so below those
  // of later rounds
  for (int i0 = h.first; i0 < h.out; i0 += kRows * kU) {
    uint4 v[kU];
    bool there[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int i = i0 + u * kRows + static_cast<int>(threadIdx.x) / kLanes;
      there[u] = false;
      if (i < h.out) {
        const uint16_t* const from = place(table, kept[i]);
        there[u] = from != nullptr;
        if (from) v[u] = *reinterpret_cast<const uint4*>(from);
      }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (there[u]) {
        uint16_t* const at = place(to, i0 + u * kRows + static_cast<int>(threadIdx.x) / kLanes);
        if (at) *reinterpret_cast<uint4*>(at) = v[u];
      }
    }
  }
}

}  // namespace fa
