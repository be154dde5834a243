// fa_weights_kernel.cuh -- the attention weight that cached keys gather from the
// new tokens' rows, found again from the LSE of the attention over the cache.
//
// Row r of a (sequence, K/V head) is token t = r % T of query head r / T of its
// group.  For every key j,
//   W'[j] = decay W[j] + sum_r [row r sees j] exp(scale q_r . k_j - LSE_r),
// with 0 for W[j] where j is a new token.  With the LSE known the sum of a key
// needs nothing of the other keys: a key belongs to one warp, which meets all its
// rows, so there are no parts to join, no atomics, and results repeat bit for bit.
#pragma once

#include "fa_paged_kernel.cuh"

namespace fa {

struct WeightsParams {
  PagedParams s;         // q, lse, table, lengths, sizes, window, scale_log2, status
  const uint16_t* k;     // [n_pages, Hk, page, D] by its strides
  long long k_page, k_head, k_token;
  float* w;              // [n_pages, Hk, page], slots contiguous
  long long w_page, w_head;
  float decay;           // 1: keys that no row sees are left alone; 0: old values are not read
};

// The keys [lo, hi) of a sequence whose weights change.
__device__ __forceinline__ SeqKeys weight_keys(const WeightsParams& p, int b) {
  SeqKeys s = seq_keys(p.s, b);
  if (p.decay != 1.f) s.lo = 0;
  return s;
}

constexpr int kWeightTile = 128;  // keys of a unit

// A CTA's share of the line of (sequence, K/V head, tile of keys) units.
struct WeightsWalk {
  long long left;  // units still to come, this one among them
  int b, hk, tile; // tile: of the sequence's
  int tile0, n;    // first tile of the sequence's keys and their number
  SeqKeys s;
};
__device__ __forceinline__ void weights_enter(const WeightsParams& p, WeightsWalk& w) {
  for (;; ++w.b) {
    w.s = weight_keys(p, w.b);
    w.tile0 = w.s.lo / kWeightTile;
    w.n = tiles_of(w.s.lo, w.s.hi, kWeightTile);
    if (w.n > 0 || w.b + 1 >= p.s.B) return;
  }
}
__device__ __forceinline__ bool weights_next(const WeightsParams& p, WeightsWalk& w) {
  if (--w.left <= 0) return false;
  if (++w.tile == w.n) {
    w.tile = 0;
    if (++w.hk == p.s.Hk) {
      w.hk = 0;
      ++w.b;
      weights_enter(p, w);
    }
  }
  return true;
}
// Block-wide; false: no units.  scratch: shared, THREADS / 32 + 2.
template <int THREADS>
__device__ __forceinline__ bool weights_share(const WeightsParams& p, long long* scratch, WeightsWalk& w) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kWarps = THREADS / 32;
  long long g = 0, gend = 0;
  for (int pass = 0; pass < 2; ++pass) {  // 0: all units, 1: the sequence that holds the share's first
    long long run = 0;
    for (int b0 = 0; b0 < p.s.B; b0 += THREADS) {
      const int b = b0 + static_cast<int>(threadIdx.x);
      long long mine = 0;
      if (b < p.s.B) {
        const SeqKeys s = weight_keys(p, b);
        mine = static_cast<long long>(p.s.Hk) * tiles_of(s.lo, s.hi, kWeightTile);
        if (pass == 0 && blockIdx.x == 0 && coherent(p.s.lens + b) > p.s.capacity) atomicOr(p.s.status, kPagedPage);
      }
      long long incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
      }
      if (lane == 31) scratch[warp] = incl;
      __syncthreads();
      long long before = run, all = 0;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        if (i < warp) before += scratch[i];
        all += scratch[i];
      }
      const long long first = before + incl - mine;
      if (pass == 1 && mine > 0 && first <= g && g < first + mine) {
        scratch[kWarps] = b;
        scratch[kWarps + 1] = first;
      }
      run += all;
      __syncthreads();
    }
    if (pass == 0) {
      g = cta_start(run, gridDim.x, blockIdx.x);
      gend = cta_start(run, gridDim.x, blockIdx.x + 1ll);
      if (g >= gend) return false;
    }
  }
  w.b = static_cast<int>(scratch[kWarps]);
  w.left = gend - g;
  weights_enter(p, w);
  const long long in = g - scratch[kWarps + 1];
  w.hk = static_cast<int>(quotient(in, w.n));
  w.tile = static_cast<int>(in - static_cast<long long>(w.hk) * w.n);
  return true;
}

// ---------------------------------------------------------------------------
// Warp-level MMAs: S^T = K Q^T, 32 keys of a tile to a warp, 8 rows at a time.
// ---------------------------------------------------------------------------
// K goes from global memory straight into the A fragments: lane 4 g + t reads 16
// bytes (8 elements) of keys g, g + 8, ... at element 32 i + 8 t, and Q's rows are
// read at the same elements for the B fragments.  A product over d may take its
// elements in any order as long as both sides agree, so no shuffle, shared memory
// or barrier stands between load and product.
constexpr int kWeightThreads = 128;

template <int D>
__global__ void __launch_bounds__(kWeightThreads, 3) fa_kv_weights_kernel(const WeightsParams p) {
  constexpr int kI = D / 32;
  __shared__ long long scratch[kWeightThreads / 32 + 2];
  grid_wait();
  grid_release();
  WeightsWalk w;
  if (!weights_share<kWeightThreads>(p, scratch, w)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g8 = lane >> 2, q4 = lane & 3;
  const int rows = p.s.rows;
  do {
    const int k0 = (w.tile0 + w.tile) * kWeightTile + warp * 32;
    if (k0 >= w.s.hi || k0 + 32 <= w.s.lo) continue;
    // 32 keys lie in one page or, of 16 tokens, in two
    const int* const table = p.s.table + static_cast<long long>(w.b) * p.s.max_pages;
    long long page[2];
    bool there[2];
    const uint16_t* src[2];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const int k = k0 + 16 * m;
      there[m] = k < w.s.hi && k + 16 > w.s.lo;
      page[m] = there[m] ? coherent(table + (k >> p.s.page_shift)) : 0;
      if (there[m] && (page[m] < 0 || page[m] >= p.s.n_pages)) {
        if (lane == 0) atomicOr(p.s.status, kPagedPage);
        there[m] = false;
      }
      if (!there[m]) page[m] = 0;
      src[m] = p.k + page[m] * p.k_page + w.hk * p.k_head + (k & ((1 << p.s.page_shift) - 1)) * p.k_token + 8 * q4;
    }
    uint4 kr[2][2][kI];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < kI; ++i)
          kr[m][h][i] = there[m] ? *reinterpret_cast<const uint4*>(src[m] + (g8 + 8 * h) * p.k_token + 32 * i)
                                 : make_uint4(0u, 0u, 0u, 0u);
    // old weights of this lane's keys (lanes with q4 == 0 write them)
    float* at[2][2];
    float old[2][2];
    bool mine[2][2];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int key = k0 + 16 * m + 8 * h + g8;
        mine[m][h] = q4 == 0 && there[m] && key >= w.s.lo && key < w.s.hi;
        at[m][h] = p.w + page[m] * p.w_page + w.hk * p.w_head + (key & ((1 << p.s.page_shift) - 1));
        old[m][h] = 0.f;
        if (mine[m][h] && p.decay != 0.f && key < w.s.len - w.s.fresh) old[m][h] = p.decay * *at[m][h];
      }
    const long long row0 = (static_cast<long long>(w.b) * p.s.Hk + w.hk) * rows;
    float sum[2][2] = {};
    for (int r0 = 0; r0 < rows; r0 += 8) {
      // this lane's two rows as columns of S^T
      int lo[2], hi[2];
      float l2[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = r0 + 2 * q4 + c;
        lo[c] = hi[c] = 0;
        l2[c] = 0.f;
        if (r < rows) {
          row_own_keys(p.s, w.s, r % p.s.T, lo[c], hi[c]);
          const float lse = p.s.lse[row0 + r];
          if (lse == -__int_as_float(0x7f800000)) hi[c] = 0;  // a row without a key
          l2[c] = lse * 1.44269504f;
        }
      }
      const bool some = (lo[0] < min(hi[0], k0 + 32) && hi[0] > k0) || (lo[1] < min(hi[1], k0 + 32) && hi[1] > k0);
      if (!__any_sync(0xffffffffu, some)) continue;
      uint4 qr[kI];
      const bool row = r0 + g8 < rows;
#pragma unroll
      for (int i = 0; i < kI; ++i)
        qr[i] = row ? *reinterpret_cast<const uint4*>(p.s.q + (row0 + r0 + g8) * D + 32 * i + 8 * q4)
                    : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < kI; ++i) {
          const uint32_t a0[4] = {kr[m][0][i].x, kr[m][1][i].x, kr[m][0][i].y, kr[m][1][i].y};
          const uint32_t a1[4] = {kr[m][0][i].z, kr[m][1][i].z, kr[m][0][i].w, kr[m][1][i].w};
          mma16816(c, a0, qr[i].x, qr[i].y);
          mma16816(c, a1, qr[i].z, qr[i].w);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = k0 + 16 * m + 8 * (e >> 1) + g8;
          const float x = ex2(fmaf(c[e], p.s.scale_log2, -l2[e & 1]));
          sum[m][e >> 1] += key >= lo[e & 1] && key < hi[e & 1] ? x : 0.f;
        }
      }
    }
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float v = sum[m][h];
        v += __shfl_xor_sync(0xffffffffu, v, 1);
        v += __shfl_xor_sync(0xffffffffu, v, 2);
        if (mine[m][h]) *at[m][h] = old[m][h] + v;
      }
  } while (weights_next(p, w));
}

// ---------------------------------------------------------------------------
// More rows: S^T = K Q^T on the tensor cores, keys on TMEM lanes.
// ---------------------------------------------------------------------------
// A CTA takes units (128 keys of one sequence and K/V head) a grid apart and streams
// past each the row blocks (128 rows) of which some row sees some of its keys.  A
// thread owns a key, so its sum stays in registers over all blocks: exponential
// and sum need no other lane.
//   warps 0-3  one key per lane: exponentials of two S buffers in turn, the sum, the
//              weight written
//   warp 4     TMA: a ring of tiles, each unit's K and then its row blocks of Q
//   warp 5     MMA
//   warp 6     the rows' LSE (times -log2 e) and bounds, beside each S buffer
// Two CTAs share an SM, so that one's products run under the other's exponentials
// also where a unit begins or ends.
// Rows that do not exist, hold no token or have lse = -inf, and keys that some row of the
// block does not see, are masked element by element (their Q may hold anything); a
// block without any takes the path without masks.
template <int D>
struct WTileCfg {
  static constexpr int kThreads = 224, kWarpProd = 4, kWarpMma = 5, kWarpSide = 6;
  static constexpr int kBoxes = D / 64;
  static constexpr uint32_t kBox = 128u * 128u;
  static constexpr uint32_t kTileBytes = kBoxes * kBox;  // 128 rows of K or Q
  static constexpr int kRing = D == 128 ? 3 : 6;
  static constexpr int kPiece = 32;                      // rows of a box of Q
  static constexpr uint32_t kSideBytes = 3 * 512 + 16;   // -L, first key, last key + 1 of 128 rows; masks wanted
  static constexpr uint32_t kSideOff = kRing * kTileBytes;
  static constexpr uint32_t kBarOff = kSideOff + 2 * kSideBytes;
  static constexpr uint32_t kTmemSlot = kBarOff + (6 + 2 * kRing + 1) * 8;
  static constexpr uint32_t kAbort = kTmemSlot + 4;
  static constexpr uint32_t kSmemBytes = kAbort + 4;
  static constexpr uint32_t kTmemCols = 256;
  static_assert(kBarOff % 8 == 0 && kSideBytes % 16 == 0, "alignment");
  static_assert(2 * (kSmemBytes + 1024) <= 233472, "two CTAs per SM");
};

// (d0, d1) = (a0 * b + c0, a1 * b + c1) as one packed f32x2 FMA
__device__ __forceinline__ void fma2c(float& d0, float& d1, float a0, float a1, float b, float c0, float c1) {
  asm("{\n\t.reg .b64 x, y, z, w;\n\t"
      "mov.b64 x, {%2, %3};\n\t"
      "mov.b64 y, {%4, %4};\n\t"
      "mov.b64 z, {%5, %6};\n\t"
      "fma.rn.f32x2 w, x, y, z;\n\t"
      "mov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b), "f"(c0), "f"(c1));
}

// The slots of the ring as the producer and the MMA issuer both see them: a tile takes the slot that was given up
// longest ago.  A row block gives its slot up at once (in the order of use), K's is kept until its unit ends, so a
// plain ring would run into it.
struct WSlots {
  uint32_t queue, phase;  // 4 bits a slot, the next one lowest; a bit per slot: parity of its uses
  int n;
  __device__ __forceinline__ explicit WSlots(int ring) : queue(0x76543210u), phase(0u), n(ring) {}
  __device__ __forceinline__ int take(uint32_t& parity) {
    const int s = static_cast<int>(queue & 15u);
    queue >>= 4;
    --n;
    parity = (phase >> s) & 1u;
    phase ^= 1u << s;
    return s;
  }
  __device__ __forceinline__ void give(int s) {
    queue = (queue & ((1u << (4 * n)) - 1u)) | (static_cast<uint32_t>(s) << (4 * n));
    ++n;
  }
};

// The units of a CTA: its number and every gridDim.x-th after it.  Whole converged warps.
struct WTileWalk {
  long long u, first;  // unit; first unit of its sequence
  int b, hk, k0;       // k0: first key of the tile
  SeqKeys s;
  int ta, tb;          // tokens that see some key of the tile
  int n;               // tiles of a head of the sequence
};
__device__ __forceinline__ bool wtile_find(const WeightsParams& p, WTileWalk& w, int b_from, long long first) {
  const int lane = threadIdx.x & 31;
  for (int b0 = b_from; b0 < p.s.B; b0 += 32) {
    SeqKeys s = {};
    int n = 0;
    if (b0 + lane < p.s.B) {
      s = weight_keys(p, b0 + lane);
      n = tiles_of(s.lo, s.hi, kWeightTile);
    }
    const long long mine = static_cast<long long>(p.s.Hk) * n;
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    const unsigned past = __ballot_sync(0xffffffffu, w.u < first + incl);
    if (past) {
      const int at = __ffs(past) - 1;
      w.b = b0 + at;
      w.first = first + __shfl_sync(0xffffffffu, incl - mine, at);
      w.n = __shfl_sync(0xffffffffu, n, at);
      w.s.len = __shfl_sync(0xffffffffu, s.len, at);
      w.s.fresh = __shfl_sync(0xffffffffu, s.fresh, at);
      w.s.lo = __shfl_sync(0xffffffffu, s.lo, at);
      w.s.hi = __shfl_sync(0xffffffffu, s.hi, at);
      return true;
    }
    first += __shfl_sync(0xffffffffu, incl, 31);
  }
  return false;
}
__device__ __forceinline__ void wtile_place(const WeightsParams& p, WTileWalk& w) {
  const long long in = w.u - w.first;
  w.hk = static_cast<int>(quotient(in, w.n));
  w.k0 = (w.s.lo / kWeightTile + static_cast<int>(in - static_cast<long long>(w.hk) * w.n)) * kWeightTile;
  const long long base = static_cast<long long>(w.s.len) - w.s.fresh;
  const int k1 = min(w.k0 + kWeightTile, w.s.hi);
  long long ta = 0, tb = w.s.fresh;
  if (p.s.right >= 0) ta = max(ta, w.k0 - base - p.s.right);
  if (p.s.left >= 0) tb = min(tb, k1 - base + p.s.left);
  w.ta = static_cast<int>(min(ta, static_cast<long long>(w.s.fresh)));
  w.tb = static_cast<int>(max(tb, 0ll));
}
__device__ __forceinline__ bool wtile_begin(const WeightsParams& p, WTileWalk& w) {
  w.u = blockIdx.x;
  if (!wtile_find(p, w, 0, 0)) return false;
  wtile_place(p, w);
  return true;
}
__device__ __forceinline__ bool wtile_next(const WeightsParams& p, WTileWalk& w) {
  w.u += gridDim.x;
  const long long end = w.first + static_cast<long long>(p.s.Hk) * w.n;
  if (w.u >= end && !wtile_find(p, w, w.b + 1, end)) return false;
  wtile_place(p, w);
  return true;
}
// Rows of the block of rows r0 .. of which some row sees some key of the tile; 0: none does.
__device__ __forceinline__ int wtile_rows(const WeightsParams& p, const WTileWalk& w, int r0) {
  const int r1 = min(p.s.rows, r0 + 128) - 1, g0 = r0 / p.s.T, g1 = r1 / p.s.T;
  const int t0 = r0 - g0 * p.s.T, t1 = r1 - g1 * p.s.T;
  bool seen;
  if (g0 == g1) seen = t0 < w.tb && t1 >= w.ta;
  else seen = w.ta < w.tb && (g1 > g0 + 1 || t0 < w.tb || t1 >= w.ta);
  return seen && w.ta < w.tb ? r1 - r0 + 1 : 0;
}

template <int D>
__global__ void __launch_bounds__(WTileCfg<D>::kThreads, 2)
    fa_kv_weights_tile_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmQ,
                              const WeightsParams p) {
  using C = WTileCfg<D>;
  extern __shared__ __align__(1024) uint8_t wtile_smem[];
  const uint32_t base = smem_addr(wtile_smem);  // 1024-byte aligned: the kernel has no static shared memory
  const uint32_t bar0 = base + C::kBarOff;
  auto bar = [&](int i) -> uint32_t { return bar0 + 8u * static_cast<uint32_t>(i); };
  // 0, 1: S written; 2, 3: S and its side buffer read; 4, 5: side buffer written; then the ring; then the drain
  auto s_full = [&](int i) -> uint32_t { return bar(i); };
  auto s_free = [&](int i) -> uint32_t { return bar(2 + i); };
  auto side_full = [&](int i) -> uint32_t { return bar(4 + i); };
  auto full = [&](int i) -> uint32_t { return bar(6 + i); };
  auto empty = [&](int i) -> uint32_t { return bar(6 + C::kRing + i); };
  const uint32_t drain = bar(6 + 2 * C::kRing);
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(wtile_smem + C::kTmemSlot);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(wtile_smem + C::kAbort);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto failed = [&](unsigned role) {
    *abort_flag = 1;
    if (lane == 0) atomicOr(p.s.status, kPagedTimeout | (role << 8));
  };
  auto uniform = [](bool v) -> bool { return __all_sync(0xffffffffu, v); };

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full(i), 1);
      mbar_init(s_free(i), 128);
      mbar_init(side_full(i), 32);
    }
    for (int i = 0; i < C::kRing; ++i) {
      mbar_init(full(i), 1);
      mbar_init(empty(i), 1);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    mbar_init_fence();
    tma_prefetch_map(&tmK);
    tma_prefetch_map(&tmQ);
  }
  grid_wait();
  grid_release();
  if (base & 1023u) {  // the swizzled layouts need it; the launch places it so
    if (threadIdx.x == 0) atomicOr(p.s.status, kPagedTimeout | (16u << 8));
    return;
  }
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < p.s.B; b += C::kThreads)
      if (coherent(p.s.lens + b) > p.s.capacity) atomicOr(p.s.status, kPagedPage);
  WTileWalk w;
  if (!wtile_begin(p, w)) return;  // the same for every warp
  if (warp == C::kWarpMma) {
    tmem_alloc(smem_addr(tmem_slot), C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int rows = p.s.rows;

  if (warp == C::kWarpProd) {
    // ======================= TMA producer =================================
    const int chunk = min(1 << p.s.page_shift, kWeightTile);  // keys of one box
    const int piece = lane / C::kBoxes, x = lane % C::kBoxes;
    WSlots slots(C::kRing);
    uint32_t used = 0;  // slots with a copy in flight or landed
    bool ok = true;
    auto take = [&]() -> int {  // the next slot, once it is free
      uint32_t parity;
      const int s = slots.take(parity);
      ok = uniform(mbar_wait(empty(s), parity ^ 1u, abort_flag));
      if (!ok) slots.phase ^= 1u << s;  // no copy was issued
      else used |= 1u << s;
      return s;
    };
    do {
      int k_slot = -1;
      for (int r0 = 0; r0 < rows; r0 += 128) {
        const int n = wtile_rows(p, w, r0);
        if (n == 0) continue;
        if (k_slot < 0) {
          const int key = w.k0 + piece * chunk;
          const bool load = lane < kWeightTile / chunk * C::kBoxes && key < w.s.hi && key + chunk > w.s.lo;
          int page = -1;
          if (load) {
            page = coherent(p.s.table + static_cast<long long>(w.b) * p.s.max_pages + (key >> p.s.page_shift));
            if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.s.n_pages)) atomicOr(p.s.status, kPagedPage);
          }
          const unsigned boxes = __popc(__ballot_sync(0xffffffffu, load));
          k_slot = take();
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(full(k_slot), boxes * chunk * 128u);
          __syncwarp();
          if (load)
            tma_load_4d(base + k_slot * C::kTileBytes + x * C::kBox + piece * chunk * 128, &tmK, full(k_slot), x * 64,
                        key & ((1 << p.s.page_shift) - 1), w.hk, page);
        }
        const int s = take();
        if (!ok) break;
        const int pieces = (n + C::kPiece - 1) / C::kPiece;
        if (lane == 0) mbar_arrive_expect_tx(full(s), pieces * C::kBoxes * C::kPiece * 128u);
        __syncwarp();
        if (lane < pieces * C::kBoxes)
          tma_load_3d(base + s * C::kTileBytes + x * C::kBox + piece * C::kPiece * 128, &tmQ, full(s), x * 64,
                      static_cast<int>((static_cast<long long>(w.b) * p.s.Hk + w.hk) * rows) + r0 + piece * C::kPiece, 0);
        slots.give(s);
      }
      if (k_slot >= 0) slots.give(k_slot);
    } while (ok && wtile_next(p, w));
    if (!ok) failed(2u);
    if (*abort_flag) {  // let every copy issued land before the CTA's shared memory goes
      for (int s = 0; s < C::kRing; ++s)
        if ((used >> s) & 1u) uniform(mbar_wait(full(s), ((slots.phase >> s) & 1u) ^ 1u, nullptr));
    }
  } else if (warp == C::kWarpMma) {
    // ======================= MMA issuer ===================================
    const uint64_t ring = sdesc_sw128(base, 16, 1024);
    WSlots slots(C::kRing);
    int block = 0;
    bool ok = true;
    auto take = [&]() -> int {  // the next tile's slot, once it has landed
      uint32_t parity;
      const int s = slots.take(parity);
      ok = uniform(mbar_wait(full(s), parity, abort_flag));
      return s;
    };
    do {
      int k_slot = -1;
      for (int r0 = 0; r0 < rows; r0 += 128) {
        const int n = wtile_rows(p, w, r0);
        if (n == 0) continue;
        if (k_slot < 0) k_slot = take();
        if (!ok) break;
        const int q_slot = take(), buf = block & 1;
        ok = ok && uniform(mbar_wait(s_free(buf), ((block >> 1) & 1) ^ 1u, abort_flag));
        if (!ok) break;
        tc_fence_after();
        const uint32_t idesc = idesc_bf16(128, (n + 31) & ~31, false);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * C::kBox + (kk & 3) * 32;
          mma_ss_elect(tmem + buf * 128, ring + ((k_slot * C::kTileBytes + off) >> 4),
                       ring + ((q_slot * C::kTileBytes + off) >> 4), idesc, kk > 0 ? 1u : 0u);
        }
        mma_commit_elect(empty(q_slot));
        mma_commit_elect(s_full(buf));
        slots.give(q_slot);
        ++block;
      }
      if (ok && k_slot >= 0) {
        mma_commit_elect(empty(k_slot));
        slots.give(k_slot);
      }
    } while (ok && wtile_next(p, w));
    if (!ok) failed(4u);
    mma_commit_elect(drain);
    uniform(mbar_wait(drain, 0, nullptr));
  } else if (warp == C::kWarpSide) {
    // ======================= LSE and bounds of the rows ====================
    int block = 0;
    bool ok = true;
    do {
      const long long row0 = (static_cast<long long>(w.b) * p.s.Hk + w.hk) * rows;
      const int k1 = min(w.k0 + kWeightTile, w.s.hi);
      for (int r0 = 0; ok && r0 < rows; r0 += 128) {
        const int n = wtile_rows(p, w, r0);
        if (n == 0) continue;
        float l2[4];
        int lo[4], hi[4];
        bool cut = (n & 31) != 0;  // columns are taken 32 at a time
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = r0 + 4 * lane + i;
          lo[i] = hi[i] = 0;
          l2[i] = 0.f;
          if (r < rows) {
            row_own_keys(p.s, w.s, r % p.s.T, lo[i], hi[i]);
            const float lse = p.s.lse[row0 + r];
            if (lse == -__int_as_float(0x7f800000)) hi[i] = 0;  // a row without a key
            l2[i] = lse * -1.44269504f;
            cut = cut || lo[i] > w.k0 || hi[i] < k1;
          }
        }
        cut = !uniform(!cut);
        const int buf = block & 1;
        if (!(ok = uniform(mbar_wait(s_free(buf), ((block >> 1) & 1) ^ 1u, abort_flag)))) break;
        uint8_t* const side = wtile_smem + C::kSideOff + buf * C::kSideBytes;
        reinterpret_cast<float4*>(side)[lane] = make_float4(l2[0], l2[1], l2[2], l2[3]);
        reinterpret_cast<int4*>(side + 512)[lane] = make_int4(lo[0], lo[1], lo[2], lo[3]);
        reinterpret_cast<int4*>(side + 1024)[lane] = make_int4(hi[0], hi[1], hi[2], hi[3]);
        if (lane == 0) *reinterpret_cast<int*>(side + 1536) = cut;
        mbar_arrive(side_full(buf));
        ++block;
      }
    } while (ok && wtile_next(p, w));
    if (!ok) failed(32u);
  } else {
    // ======================= exponentials and sums =========================
    const uint32_t lanes = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    const float c = p.s.scale_log2;
    int block = 0;
    bool ok = true;
    do {
      const int key = w.k0 + warp * 32 + lane;
      float* at = nullptr;
      float old = 0.f;
      if (key >= w.s.lo && key < w.s.hi) {
        const int page = coherent(p.s.table + static_cast<long long>(w.b) * p.s.max_pages + (key >> p.s.page_shift));
        if (static_cast<unsigned>(page) < static_cast<unsigned>(p.s.n_pages)) {
          at = p.w + page * p.w_page + w.hk * p.w_head + (key & ((1 << p.s.page_shift) - 1));
          if (p.decay != 0.f && key < w.s.len - w.s.fresh) old = p.decay * *at;
        } else {
          atomicOr(p.s.status, kPagedPage);
        }
      }
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
      for (int r0 = 0; ok && r0 < rows; r0 += 128) {
        const int n = wtile_rows(p, w, r0);
        if (n == 0) continue;
        const int buf = block & 1;
        const uint32_t ph = (block >> 1) & 1;
        ok = uniform(mbar_wait(side_full(buf), ph, abort_flag) && mbar_wait(s_full(buf), ph, abort_flag));
        if (!ok) break;
        tc_fence_after();
        const uint8_t* const side = wtile_smem + C::kSideOff + buf * C::kSideBytes;
        const bool cut = *reinterpret_cast<const int*>(side + 1536) != 0;
#pragma unroll 1
        for (int g = 0; g < n; g += 32) {
          uint32_t r[32];
          tmem_ld32(lanes + buf * 128 + g, r);
          const float4* const l4 = reinterpret_cast<const float4*>(side) + g / 4;
          tmem_ld_wait(r);
          float* const f = reinterpret_cast<float*>(r);
          if (!cut) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 l = l4[i];
              float x0, x1, x2, x3;
              fma2c(x0, x1, f[4 * i], f[4 * i + 1], c, l.x, l.y);
              fma2c(x2, x3, f[4 * i + 2], f[4 * i + 3], c, l.z, l.w);
              add2(sum[0], sum[1], ex2(x0), ex2(x1));
              add2(sum[2], sum[3], ex2(x2), ex2(x3));
            }
          } else {
            const int4* const lo4 = reinterpret_cast<const int4*>(side + 512) + g / 4;
            const int4* const hi4 = reinterpret_cast<const int4*>(side + 1024) + g / 4;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 l = l4[i];
              const int4 lo = lo4[i], hi = hi4[i];
              float x0, x1, x2, x3;
              fma2c(x0, x1, f[4 * i], f[4 * i + 1], c, l.x, l.y);
              fma2c(x2, x3, f[4 * i + 2], f[4 * i + 3], c, l.z, l.w);
              x0 = key >= lo.x && key < hi.x ? ex2(x0) : 0.f;
              x1 = key >= lo.y && key < hi.y ? ex2(x1) : 0.f;
              x2 = key >= lo.z && key < hi.z ? ex2(x2) : 0.f;
              x3 = key >= lo.w && key < hi.w ? ex2(x3) : 0.f;
              add2(sum[0], sum[1], x0, x1);
              add2(sum[2], sum[3], x2, x3);
            }
          }
        }
        tc_fence_before();
        mbar_arrive(s_free(buf));
        ++block;
      }
      if (!ok) break;
      if (at) *at = old + ((sum[0] + sum[1]) + (sum[2] + sum[3]));
    } while (wtile_next(p, w));
    if (!ok) failed(1u);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == C::kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

}  // namespace fa
