// fa_evict_kernel.cuh -- the keys of a paged cache that gathered the least weight
// leave it, and the others move together.
//
// A sequence of len > budget + slack tokens keeps `budget` of them, for every K/V
// head its own: the first `sinks`, the last `recent`, and of those between the
// heaviest (of equal ones the lower slots).  They keep their order, so the i-th of
// them goes to slot i, which is never above its own.
//   fa_evict_select_kernel  per (sequence, K/V head): the list of kept slots, by a
//     radix selection of the smallest kept weight (few heads of many weights:
//     fa_evict_count_kernel for each digit, fa_evict_list_kernel);
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

struct EvictFound {  // the search for the smallest kept weight, per (sequence, K/V head) and digit
  unsigned prefix;   // its digits so far
  int want;          // how many of the weights that share them stay
  int all;           // all of those: the search is over
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
  EvictFound* found;     // the selection in parts: [2, B Hk], after one digit and two
  int* above;            // [B Hk, split]: weights of a part that stay by the digits so far
  int* hist;             // [2, B Hk, split, kSelectBins]: a part's counts, of digits 0 and 2, and 1
  int split;             // parts of a head's weights
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

// Selection: the smallest kept weight is found by its bits, 11 + 11 + 10 of them from
// the top: a histogram of the free weights that share the bits so far, and the digit at
// which the kept ones run out.  11 bits first (sign, exponent, two of the fraction),
// because weights share exponents: with 8 most counts of a warp met in the same few
// words.  It ends early where all weights of that digit stay, after two digits as a
// rule.  Then every warp counts what stays in its part of the list, and after one sum
// over the warps writes it, in order.  A thread takes four weights at a time everywhere.
constexpr int kSelectBins = 2048;
__device__ constexpr int digit_shift(int digit) { return digit == 0 ? 21 : (digit == 1 ? 10 : 0); }
__device__ constexpr unsigned digit_mask(int digit) { return digit == 2 ? 0x3ffu : 0x7ffu; }
// order ^ prefix of a weight that shares the digits before has none but these bits
__device__ constexpr unsigned digit_rest(int digit) { return digit == 0 ? 0xffffffffu : (digit == 1 ? 0x1fffffu : 0x3ffu); }

// What the selection needs of one (sequence, K/V head).
struct SelectHead {
  const int* table;
  const float* w;
  int* kept;
  int raw, len, out;  // as given, within the table, afterwards
  int lo, hi;         // the free ones
  int want;           // how many of them stay
  bool over;          // more than may stay
  __device__ __forceinline__ SelectHead(const EvictParams& p, int bh) {
    const int b = bh / p.Hk;
    table = p.table + static_cast<long long>(b) * p.max_pages;
    w = p.w + bh % p.Hk * p.w_head;
    kept = p.kept + static_cast<long long>(bh) * p.most;
    raw = coherent(p.lens + b);
    len = max(0, min(raw, p.capacity));
    over = len > p.most;
    out = over ? p.budget : len;
    lo = p.sinks;
    hi = len - p.recent;
    want = p.budget - p.sinks - p.recent;
  }
};

// f(j, weights of tokens w0 + j .. w0 + j + 3) for the multiples of four j < n, whatever thread takes them; w0 is a
// multiple of 16, and four tokens lie in one page.  Those past n are undefined.
template <int THREADS, typename F>
__device__ __forceinline__ void for_weights(const EvictParams& p, const SelectHead& h, int w0, int n, F f) {
  const int mask = (1 << p.page_shift) - 1;
  constexpr int kU = 4;  // in flight
  for (int j0 = 4 * static_cast<int>(threadIdx.x); j0 < n; j0 += 4 * kU * THREADS) {
    int page[kU];
    float4 v[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int j = j0 + 4 * u * THREADS;
      page[u] = j < n ? coherent(h.table + ((w0 + j) >> p.page_shift)) : 0;
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
      const float* const at = h.w + page[u] * p.w_page + ((w0 + j) & mask);
      if (p.w_vec) {
        const uint4 x = load16(reinterpret_cast<const uint16_t*>(at));
        v[u] = make_float4(__uint_as_float(x.x), __uint_as_float(x.y), __uint_as_float(x.z), __uint_as_float(x.w));
      } else {
        v[u] = make_float4(load4(at), load4(at + 1), load4(at + 2), load4(at + 3));
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if (j0 + 4 * u * THREADS < n) f(j0 + 4 * u * THREADS, v[u]);
  }
}

// Counts those of four weights, of which j0 <= j < j1 are free, that share the digits before `digit`.
__device__ __forceinline__ void count_digit(int* hist, int digit, unsigned prefix, int j, int j0, int j1,
                                            const float4& v) {
  const unsigned o[4] = {weight_order(v.x), weight_order(v.y), weight_order(v.z), weight_order(v.w)};
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (j + e >= j0 && j + e < j1 && (o[e] ^ prefix) <= digit_rest(digit))
      atomicAdd(&hist[(o[e] >> digit_shift(digit)) & digit_mask(digit)], 1);
}

// The bins of thread t run from kSelectBins - 1 - t * (bins each) downwards, so that sums run from the heaviest.
template <int THREADS>
__device__ __forceinline__ int select_bin(int i) {
  return kSelectBins - 1 - kSelectBins / THREADS * static_cast<int>(threadIdx.x) - i;
}

// The digit at which `want` weights are reached, from this thread's bins; block-wide, begins and ends in a barrier.
// Shared: found[3] (digit, how many of its weights stay, how many there are), counts[32].
template <int THREADS>
__device__ __forceinline__ void find_digit(const int (&n)[kSelectBins / THREADS], int want, int* counts, int* found) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int all = 0;
#pragma unroll
  for (int i = 0; i < kSelectBins / THREADS; ++i) all += n[i];
  int incl = all;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += up;
  }
  __syncthreads();
  if (lane == 31) counts[warp] = incl;
  __syncthreads();
  int above = __reduce_add_sync(0xffffffffu, lane < warp ? counts[lane] : 0) + incl - all;
  if (above < want && want <= above + all) {
#pragma unroll
    for (int i = 0; i < kSelectBins / THREADS; ++i) {
      if (above < want && want <= above + n[i]) {
        found[0] = select_bin<THREADS>(i);
        found[1] = want - above;
        found[2] = n[i];
      }
      above += n[i];
    }
  }
  __syncthreads();
}

// The list of tokens [w0, w0 + n), whose weights are in vals, behind `heavier` kept ones that stay for sure and `equal`
// others with the smallest kept weight, of which `ties` stay (below 0: all).  Block-wide, ends without a barrier;
// heavier and equal move on.
template <int THREADS>
__device__ __forceinline__ void write_list(const SelectHead& h, const float4* vals, int w0, int n, unsigned least,
                                           int ties, int& heavier, int& equal, int (&counts)[2][32], int* first_gone) {
  constexpr int kWarps = THREADS / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int part = ((n + kWarps - 1) / kWarps + 127) & ~127;  // of a warp
  const int j0 = min(n, warp * part), j1 = min(n, j0 + part);
  const int f0 = h.lo - w0, f1 = h.hi - w0;
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
  a = lane < kWarps ? counts[0][lane] : 0;
  t = lane < kWarps ? counts[1][lane] : 0;
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
      if (is_sure || (is_tie && before < ties)) {
        const int to = at + min(before, max(ties, 0));
        if (to < h.out) h.kept[to] = w0 + j + e;  // it is, unless weights change under the call
      } else if (j + e < j1) {
        gone = min(gone, w0 + j + e);
      }
      at += is_sure;
      before += is_tie;
    }
    a += all & 0xffff;
    t += all >> 16;
  }
  gone = __reduce_min_sync(0xffffffffu, gone);
  if (lane == 0) atomicMin(first_gone, gone);  // where the first one goes, the list leaves its slots
}

// One CTA to a head: its weights are brought to shared memory once (in windows where
// they are more than fit).  Bound: one SM's instructions and latency per head.  Under a
// profiler, caches cold: 128 heads of up to 8192 weights 15.6 us, 96 of up to 1024 8.4
// (with one weight to a thread 23 and 12).  A bracket from a sample of the weights
// before the first digit made 32000 weights 74 us of 54.
template <int THREADS>
__global__ void __launch_bounds__(THREADS, 1) fa_evict_select_kernel(const EvictParams p) {
  constexpr int kBinsEach = kSelectBins / THREADS;
  extern __shared__ __align__(1024) uint8_t select_smem[];
  float4* const vals = reinterpret_cast<float4*>(select_smem);  // [window / 4]
  __shared__ int hist[kSelectBins];
  __shared__ int counts[2][32];
  __shared__ int found[3];
  __shared__ int first_gone;
  grid_wait();
  grid_release();
  const int tid = static_cast<int>(threadIdx.x);
  const SelectHead h(p, blockIdx.x);
  if (h.raw > p.capacity && tid == 0) atomicOr(p.status, kPagedPage);
  const bool fork = p.table_out != p.table;
  for (int i = h.out + tid; i < p.most; i += THREADS) h.kept[i] = -1;
  if (!h.over) {  // stays as it is
    for (int i = tid; i < h.len; i += THREADS) h.kept[i] = i;
    if (tid == 0) p.heads[blockIdx.x] = {h.len, h.len, fork ? 0 : h.len, 0};
    return;
  }
  if (tid == 0) first_gone = h.out;
  auto load = [&](int w0) {
    for_weights<THREADS>(p, h, w0, min(p.window, h.len - w0), [&](int j, const float4& v) { vals[j / 4] = v; });
  };
  const int windows = (h.len + p.window - 1) / p.window;
  unsigned least = 0xffffffffu;  // the smallest order that is kept among the free ones
  int ties = 0;                  // how many of that order; below 0: all from `least` on
  bool loaded = false;
  int want = h.want;
  if (want > 0) {
    unsigned prefix = 0;
#pragma unroll 1
    for (int digit = 0; digit < 3; ++digit) {
      for (int i = tid; i < kSelectBins; i += THREADS) hist[i] = 0;
      for (int k = 0; k < windows; ++k) {
        const int w0 = k * p.window, n = min(p.window, h.len - w0);
        if (!loaded) {
          __syncthreads();  // the window before has been read
          load(w0);
        }
        __syncthreads();
        for (int j = 4 * tid; j < n; j += 4 * THREADS)
          count_digit(hist, digit, prefix, j, h.lo - w0, min(h.hi - w0, n), vals[j / 4]);
      }
      loaded = windows == 1;
      __syncthreads();
      int n[kBinsEach];
#pragma unroll
      for (int i = 0; i < kBinsEach; ++i) n[i] = hist[select_bin<THREADS>(i)];
      find_digit<THREADS>(n, want, counts[0], found);
      prefix |= static_cast<unsigned>(found[0]) << digit_shift(digit);
      want = found[1];
      if (want == found[2]) break;
    }
    least = prefix;  // zeros below the digits that were looked at
    ties = want == found[2] ? -1 : want;
  }
  int heavier = 0, equal = 0;  // kept so far without and with the order `least`, in the windows before
  for (int k = 0; k < windows; ++k) {
    const int w0 = k * p.window;
    if (!loaded) {
      __syncthreads();
      load(w0);
    }
    __syncthreads();
    write_list<THREADS>(h, vals, w0, min(p.window, h.len - w0), least, ties, heavier, equal, counts, &first_gone);
    loaded = false;
  }
  __syncthreads();
  if (tid == 0) p.heads[blockIdx.x] = {h.len, h.out, fork ? 0 : first_gone, 0};
}

// Few heads of many weights: p.split CTAs to a head, each with a part of its weights, and a
// kernel to a digit and one for the list.  Bound: four kernels' chains of dependent reads and
// barriers, about 4.5 us each.  (Parts in a cluster that read one another's counts from
// shared memory would be one launch; a kernel of that kind faulted and was taken out.  The
// move took its list's slots unchecked then, so a list with places left out would explain it.)
// A part's histogram goes to the workspace; the next kernel's CTAs each add those of their
// head up, and note what of their own part stays by the digit found, so that the last one
// knows where each part's list begins.
constexpr int kSplitThreads = 512;
constexpr int kMostParts = 16, kPartCtas = 152;  // parts of a head at most, of all heads about
inline int select_parts(long long heads) {
  const long long n = kPartCtas / heads;
  return static_cast<int>(n < kMostParts ? n : kMostParts);
}

// Written by the kernel before, which may still have read its neighbours on this SM.
__device__ __forceinline__ EvictFound load_found(const EvictFound* at) {
  const uint4 x = load16(reinterpret_cast<const uint16_t*>(at));
  return {x.x, static_cast<int>(x.y), static_cast<int>(x.z), 0};
}

struct SelectPart {
  int head, part, t0, t1;  // its tokens: equal shares in pages of 256
  __device__ __forceinline__ SelectPart(const EvictParams& p)
      : head(static_cast<int>(blockIdx.x) / p.split), part(static_cast<int>(blockIdx.x) % p.split) {}
  __device__ __forceinline__ void cut(const EvictParams& p, int len) {
    const int each = ((len + p.split - 1) / p.split + 255) & ~255;
    t0 = static_cast<int>(min(static_cast<long long>(len), static_cast<long long>(part) * each));
    t1 = min(len, t0 + each);
  }
};

// The digit before `digit`, from the parts' histograms of it; f moves on.  Also: what of the parts [from, to) is above it
// (with it where all of it stays), in `above` of every thread, and how many of them have it where not all stay.
template <int DIGIT>
__device__ __forceinline__ void join_parts(const EvictParams& p, int head, int from, int to, EvictFound& f, int& above,
                                           int& equal, int* counts, int* found) {
  constexpr int kBinsEach = kSelectBins / kSplitThreads;
  static_assert(kBinsEach == 4, "a thread's bins are four words");
  const int bin = select_bin<kSplitThreads>(kBinsEach - 1), heads = p.B * p.Hk;  // its lowest bin
  const int* const rows =
      p.hist + ((DIGIT & 1ll) * heads + head) * p.split * kSelectBins + bin;
  int n[kBinsEach] = {}, m[kBinsEach] = {};  // of all parts, of the parts [from, to); the highest bin first
#pragma unroll 4
  for (int i = 0; i < p.split; ++i) {
    const uint4 x = load16(reinterpret_cast<const uint16_t*>(rows + i * kSelectBins));
    const int c[kBinsEach] = {static_cast<int>(x.w), static_cast<int>(x.z), static_cast<int>(x.y), static_cast<int>(x.x)};
#pragma unroll
    for (int e = 0; e < kBinsEach; ++e) {
      n[e] += c[e];
      if (i >= from && i < to) m[e] += c[e];
    }
  }
  find_digit<kSplitThreads>(n, f.want, counts, found);
  f.prefix |= static_cast<unsigned>(found[0]) << digit_shift(DIGIT);
  f.want = found[1];
  f.all = found[1] == found[2];
  int a = 0, t = 0;
#pragma unroll
  for (int e = 0; e < kBinsEach; ++e) {
    const int at = bin + kBinsEach - 1 - e;
    if (at > found[0] || (f.all && at == found[0])) a += m[e];
    else if (at == found[0]) t += m[e];
  }
  a = __reduce_add_sync(0xffffffffu, a);
  t = __reduce_add_sync(0xffffffffu, t);
  __syncthreads();  // counts and found have been read
  if ((threadIdx.x & 31) == 0) {
    counts[threadIdx.x >> 5] = a;
    counts[16 + (threadIdx.x >> 5)] = t;
  }
  static_assert(kSplitThreads / 32 == 16, "two sums of 16 warps");
  __syncthreads();
  const int x = counts[threadIdx.x & 31];
  above = __reduce_add_sync(0xffffffffu, (threadIdx.x & 31) < 16 ? x : 0);
  equal = __reduce_add_sync(0xffffffffu, (threadIdx.x & 31) < 16 ? 0 : x);
}

template <int DIGIT>
__global__ void __launch_bounds__(kSplitThreads) fa_evict_count_kernel(const EvictParams p) {
  __shared__ __align__(16) int hist[kSelectBins];
  __shared__ int counts[32];
  __shared__ int found[3];
  grid_wait();
  grid_release();
  const int tid = static_cast<int>(threadIdx.x);
  SelectPart me(p);
  const SelectHead h(p, me.head);
  if (DIGIT == 0 && me.part == 0 && tid == 0) {
    if (h.raw > p.capacity) atomicOr(p.status, kPagedPage);
    p.heads[me.head] = {h.len, h.out, p.table_out != p.table ? 0 : h.out, 0};  // first: the list's parts lower it
  }
  if (!h.over || h.want == 0) return;
  for (int i = tid; i < kSelectBins; i += kSplitThreads) hist[i] = 0;
  me.cut(p, h.len);
  EvictFound f = {0u, h.want, 0, 0};
  if constexpr (DIGIT > 0) {
    const int heads = p.B * p.Hk;
    if (DIGIT == 2) f = load_found(p.found + me.head);
    if (!f.all) {
      int above, equal;
      join_parts<DIGIT - 1>(p, me.head, me.part, me.part + 1, f, above, equal, counts, found);
      if (tid == 0) p.above[blockIdx.x] = (DIGIT == 2 ? coherent(p.above + blockIdx.x) : 0) + above;
    }
    if (me.part == 0 && tid == 0) p.found[(DIGIT - 1) * heads + me.head] = f;
    if (f.all) return;
  }
  __syncthreads();
  for_weights<kSplitThreads>(p, h, me.t0, me.t1 - me.t0, [&](int j, const float4& v) {
    count_digit(hist, DIGIT, f.prefix, j, h.lo - me.t0, min(h.hi, me.t1) - me.t0, v);
  });
  __syncthreads();
  int* const row = p.hist + ((DIGIT & 1ll) * p.B * p.Hk * p.split + blockIdx.x) * kSelectBins;
  for (int i = 4 * tid; i < kSelectBins; i += 4 * kSplitThreads)
    *reinterpret_cast<int4*>(row + i) = *reinterpret_cast<const int4*>(hist + i);
}

__global__ void __launch_bounds__(kSplitThreads) fa_evict_list_kernel(const EvictParams p) {
  extern __shared__ __align__(1024) uint8_t select_smem[];
  float4* const vals = reinterpret_cast<float4*>(select_smem);  // [window / 4]
  __shared__ int counts[2][32];
  __shared__ int found[3];
  __shared__ int first_gone;
  grid_wait();
  grid_release();
  const int tid = static_cast<int>(threadIdx.x);
  SelectPart me(p);
  const SelectHead h(p, me.head);
  me.cut(p, h.len);
  if (me.part == 0)
    for (int i = h.out + tid; i < p.most; i += kSplitThreads) h.kept[i] = -1;
  if (!h.over) {  // stays as it is
    for (int i = me.t0 + tid; i < me.t1; i += kSplitThreads) h.kept[i] = i;
    return;
  }
  if (tid == 0) first_gone = 0x7fffffff;
  unsigned least = 0xffffffffu;
  int ties = 0;
  int heavier = min(me.t0, h.lo) + max(0, me.t0 - h.hi), equal = 0;  // of the parts before: those held by their places
  if (h.want > 0) {
    EvictFound f = load_found(p.found + p.B * p.Hk + me.head);
    const int before = tid < me.part ? coherent(p.above + me.head * p.split + tid) : 0;  // kMostParts threads of the first warp
    int above = 0;
    if (!f.all) join_parts<2>(p, me.head, 0, me.part, f, above, equal, counts[0], found);
    if (tid < 32) {
      const int sum = __reduce_add_sync(0xffffffffu, before);
      if (tid == 0) found[0] = sum;
    }
    __syncthreads();
    heavier += found[0] + above;
    least = f.prefix;
    ties = f.all ? -1 : f.want;
  }
  for (int w0 = me.t0; w0 < me.t1; w0 += p.window) {
    const int n = min(p.window, me.t1 - w0);
    __syncthreads();  // the window before, and counts, have been read
    for_weights<kSplitThreads>(p, h, w0, n, [&](int j, const float4& v) { vals[j / 4] = v; });
    __syncthreads();
    write_list<kSplitThreads>(h, vals, w0, n, least, ties, heavier, equal, counts, &first_gone);
  }
  __syncthreads();
  if (tid == 0 && p.table_out == p.table && first_gone < h.out) atomicMin(&p.heads[me.head].first, first_gone);
}

// The rows of K or V, or the weights, of one (sequence, K/V head), by one cluster (by any
// CTAs where they go to other pages).  A round takes
// kRows * kU rows of each CTA; all of a round are read before any is written, and as a
// destination lies at or below its own source, it lies below the sources of later
// rounds, so that one barrier of the cluster stands between a round's loads and its
// stores and nothing after them.  Into other pages no barrier is needed.
// Bound: memory; a round in place waits for its loads (a cluster has its rows of the
// next round looked up meanwhile), which shows where few rows are moved: 128 heads of up to
// 8192 halved, K and V of 128, 74 us cold (the whole call 87 on caches that L2 does not hold, 38 to
// 41 repeated on one), 16 heads of up to 31999 to 8000 into other pages 32.
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
  // within the table even where weights changed under the selection, which then left places of the list out
  auto slot_of = [&](int i) -> int {
    return static_cast<int>(min(static_cast<unsigned>(coherent(kept + i)), static_cast<unsigned>(h.len - 1)));
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
        const int slot = slot_of(i), page = page_of(table, slot);
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
      from[u] = i < h.out ? place(table, slot_of(i)) : nullptr;
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
