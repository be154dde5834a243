// fa_weights_kernel.cuh -- the attention weight that cached keys gather from the
// new tokens' rows, found again from the LSE of the attention over the cache.
//
// Row r of a (sequence, K/V head) is token t = r % T of query head r / T of its
// group.  For every key j,
//   W'[j] = decay W[j] + sum_r [row r sees j] exp(scale q_r . k_j - LSE_r),
// with 0 for W[j] where j is a new token.  With the LSE known the sum of a key
// needs nothing of the other keys.  On the warp-level kernel a key belongs to one warp,
// which meets all its rows; on the tensor cores two groups of warps, and the CTAs of a
// cluster, take row blocks in turn, and a writer joins their sums in a fixed order.
// No atomics: results repeat bit for bit.
#pragma once

#include "fa_cache_ptx.cuh"
#include "fa_paged_kernel.cuh"

namespace fa {

struct WeightsParams {
  PagedParams s;         // q, lse, table, lengths, sizes, window, scale_log2, status
  const uint16_t* k;     // [n_pages, Hk, page, D] by its strides
  long long k_page, k_head, k_token;
  float* w;              // [n_pages, Hk, page], slots contiguous
  long long w_page, w_head;
  float decay;           // 1: keys that no row sees are left alone; 0: old values are not read
  int group;                // query heads of a K/V head
  int uneven;               // units differ by many row blocks: given out by what each cluster has to do
  unsigned t_mul, t_shift;  // r / T = r * t_mul >> 32 + t_shift for the rows r < 2^31 (T > 1)
};
// Query head (in its group) of row r.
__device__ __forceinline__ int row_head(const WeightsParams& p, int r) {
  return p.s.T == 1 ? r : static_cast<int>(__umulhi(static_cast<unsigned>(r), p.t_mul) >> p.t_shift);
}

// The keys [lo, hi) of a sequence whose weights change.
__device__ __forceinline__ SeqKeys weight_keys(const WeightsParams& p, int b) {
  SeqKeys s = seq_keys(p.s, b);
  if (p.decay != 1.f) s.lo = 0;
  return s;
}

constexpr int kWeightTile = 128;  // keys of a tile of the tensor-core kernel

// A CTA's share of the line of (sequence, K/V head, tile of keys) units.
struct WeightsWalk {
  long long left;  // units still to come, this one among them
  int b, hk, tile; // tile: of the sequence's
  int tile0, n;    // first tile of the sequence's keys and their number
  SeqKeys s;
};
template <int TILE>
__device__ __forceinline__ void weights_enter(const WeightsParams& p, WeightsWalk& w) {
  for (;; ++w.b) {
    w.s = weight_keys(p, w.b);
    w.tile0 = w.s.lo / TILE;
    w.n = tiles_of(w.s.lo, w.s.hi, TILE);
    if (w.n > 0 || w.b + 1 >= p.s.B) return;
  }
}
template <int TILE>
__device__ __forceinline__ bool weights_next(const WeightsParams& p, WeightsWalk& w) {
  if (--w.left <= 0) return false;
  if (++w.tile == w.n) {
    w.tile = 0;
    if (++w.hk == p.s.Hk) {
      w.hk = 0;
      ++w.b;
      weights_enter<TILE>(p, w);
    }
  }
  return true;
}
// Block-wide; false: no units.  scratch: shared, THREADS / 32 + 2.
template <int THREADS, int TILE>
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
        mine = static_cast<long long>(p.s.Hk) * tiles_of(s.lo, s.hi, TILE);
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
  weights_enter<TILE>(p, w);
  const long long in = g - scratch[kWarps + 1];
  w.hk = static_cast<int>(quotient(in, w.n));
  w.tile = static_cast<int>(in - static_cast<long long>(w.hk) * w.n);
  return true;
}

// ---------------------------------------------------------------------------
// Warp-level MMAs: S^T = K Q^T, 16 M keys of a tile to a warp, 8 rows at a time.
// ---------------------------------------------------------------------------
// K goes from global memory straight into the A fragments: lane 4 g + t reads 16
// bytes (8 elements) of keys g, g + 8, ... at element 32 i + 8 t, and Q's rows are
// read at the same elements for the B fragments.  A product over d may take its
// elements in any order as long as both sides agree, so no shuffle, shared memory
// or barrier stands between load and product.  A warp has 8 KB of K in flight (4 KB where
// units are few), and the page indices of its next tile are read behind them.
// Bound: memory, K once and 8 bytes a key.  32 sequences of up to 8192 keys, 8 K/V heads of
// 128 under 32 query heads: 51.1 us, 5.6 TB/s (58.6 without the pages read ahead, 71 where
// the compiler may sink K's loads behind those of the old weights); 8 x up to 1024 keys, 12
// heads of 64: 4.9 us, most of it the launch and three reads in a row (length, page, K).
constexpr int kWeightThreads = 128;
template <int M>
struct WRowsCfg {
  static constexpr int kM = M;                               // fragments of 16 keys
  static constexpr int kKeys = 16 * kM;                      // keys of a warp
  static constexpr int kTile = kWeightThreads / 32 * kKeys;  // keys of a unit
};

template <int D, int M>
__global__ void __launch_bounds__(kWeightThreads, 3) fa_kv_weights_kernel(const WeightsParams p) {
  using C = WRowsCfg<M>;
  constexpr int kI = D / 32, kM = C::kM;
  __shared__ long long scratch[kWeightThreads / 32 + 2];
  grid_wait();
  grid_release();
  WeightsWalk w;
  if (!weights_share<kWeightThreads, C::kTile>(p, scratch, w)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g8 = lane >> 2, q4 = lane & 3;
  const int rows = p.s.rows;
  // 16 keys lie in one page
  auto first_key = [&](const WeightsWalk& v) -> int { return (v.tile0 + v.tile) * C::kTile + warp * C::kKeys; };
  auto wanted = [&](const WeightsWalk& v, int m) -> bool {
    const int k = first_key(v) + 16 * m;
    return k < v.s.hi && k + 16 > v.s.lo;
  };
  auto page_of = [&](const WeightsWalk& v, int m) -> int {
    return wanted(v, m) ? coherent(p.s.table + static_cast<long long>(v.b) * p.s.max_pages +
                                   ((first_key(v) + 16 * m) >> p.s.page_shift))
                        : 0;
  };
  int next_page[kM];
#pragma unroll
  for (int m = 0; m < kM; ++m) next_page[m] = page_of(w, m);
  bool more;
  do {
    const WeightsWalk u = w;
    const int k0 = first_key(u);
    long long page[kM];
    bool there[kM];
    uint4 kr[kM][2][kI];
#pragma unroll
    for (int m = 0; m < kM; ++m) {
      page[m] = next_page[m];
      there[m] = wanted(u, m);
      if (there[m] && static_cast<unsigned>(next_page[m]) >= static_cast<unsigned>(p.s.n_pages)) {
        if (lane == 0) atomicOr(p.s.status, kPagedPage);
        there[m] = false;
      }
      if (!there[m]) page[m] = 0;
      const uint16_t* const src = p.k + page[m] * p.k_page + u.hk * p.k_head +
                                  ((k0 + 16 * m) & ((1 << p.s.page_shift) - 1)) * p.k_token + 8 * q4;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < kI; ++i)
          kr[m][h][i] = there[m] ? load16(src + (g8 + 8 * h) * p.k_token + 32 * i) : make_uint4(0u, 0u, 0u, 0u);
    }
    // old weights of this lane's keys (lanes with q4 == 0 write them)
    auto key_of = [&](int m, int h) -> int { return k0 + 16 * m + 8 * h + g8; };
    auto mine = [&](int m, int h) -> bool {
      return q4 == 0 && there[m] && key_of(m, h) >= u.s.lo && key_of(m, h) < u.s.hi;
    };
    auto at = [&](int m, int h) -> float* {
      return p.w + page[m] * p.w_page + u.hk * p.w_head + (key_of(m, h) & ((1 << p.s.page_shift) - 1));
    };
    float old[kM][2];
#pragma unroll
    for (int m = 0; m < kM; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        old[m][h] = 0.f;
        if (mine(m, h) && p.decay != 0.f && key_of(m, h) < u.s.len - u.s.fresh) old[m][h] = load4(at(m, h));
      }
    more = weights_next<C::kTile>(p, w);
#pragma unroll
    for (int m = 0; m < kM; ++m) next_page[m] = more ? page_of(w, m) : 0;
    if (k0 >= u.s.hi || k0 + C::kKeys <= u.s.lo) continue;
    const long long row0 = (static_cast<long long>(u.b) * p.s.Hk + u.hk) * rows;
    float sum[kM][2] = {};
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
          row_own_keys(p.s, u.s, r - row_head(p, r) * p.s.T, lo[c], hi[c]);
          const float lse = p.s.lse[row0 + r];
          if (lse == -__int_as_float(0x7f800000)) hi[c] = 0;  // a row without a key
          l2[c] = lse * 1.44269504f;
        }
      }
      const bool some = (lo[0] < min(hi[0], k0 + C::kKeys) && hi[0] > k0) ||
                        (lo[1] < min(hi[1], k0 + C::kKeys) && hi[1] > k0);
      if (!__any_sync(0xffffffffu, some)) continue;
      uint4 qr[kI];
      const bool row = r0 + g8 < rows;
#pragma unroll
      for (int i = 0; i < kI; ++i)
        qr[i] = row ? *reinterpret_cast<const uint4*>(p.s.q + (row0 + r0 + g8) * D + 32 * i + 8 * q4)
                    : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int m = 0; m < kM; ++m) {
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
    for (int m = 0; m < kM; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float v = sum[m][h];
        v += __shfl_xor_sync(0xffffffffu, v, 1);
        v += __shfl_xor_sync(0xffffffffu, v, 2);
        if (mine(m, h)) *at(m, h) = fmaf(p.decay, old[m][h], v);
      }
  } while (more);
}

// ---------------------------------------------------------------------------
// More rows: S^T = K Q^T on the tensor cores, keys on TMEM lanes.
// ---------------------------------------------------------------------------
// A cluster takes units (256 keys of one sequence and K/V head) and streams past each
// the row blocks (128 rows) that see some of its keys; its CTAs take them in turn.  A
// thread owns a key, so its sum stays in registers over all its blocks: exponential
// and sum need no other lane.
//   warps 0-15  tile (warp / 4) % 2 of the keys, one key per lane, every other row block
//              (S buffer warp / 8): exponentials and their sum, handed to the writer at
//              a unit's end
//   warp 16    TMA: a ring of tiles, each unit's K and then its row blocks of Q
//   warp 17    MMA
//   warp 18    the rows' tokens and LSE (times -log2 e) beside each S buffer
//   warp 19    the writer, while the next unit's products run: joins the groups' sums,
//              sends them to the cluster's first CTA, and there adds all to the old weights
//              before and after that it finds the cluster's units and describes them, a few ahead
// 256 keys and one CTA to an SM: a row block, once loaded, waited for and described,
// passes two tiles (2 x 2048 tokens over 8192, 32/8 heads of 128: 169 us, with 128 keys and
// two CTAs 221; 147 us since a writer has a warp of its own, the units come described
// and the MMAs are issued with constant indexes, 142 since long units are given out by
// what each cluster has to do).
// Bound: the products (80 us at the measured tensor rate) and one exponential per key and
// row, which take turns on two buffers.  By timestamps in that case (146 us with them) a CTA
// needs 7 us to its first block (3.4 of them the search for its units), 0.77 us for a row
// block and 256 keys (0.66 of it the products at that rate), 4.6 us for a unit beside its
// blocks and 3 us after the last; the last CTA to end has 134 blocks in 7 units.
// With many row blocks the CTAs of a cluster share a unit, so that it is small beside a
// CTA's share and few keys still reach many SMs.
// Rows that do not exist, hold no token or have lse = -inf, and keys that some row of the
// block does not see, are masked element by element (their Q may hold anything): a key
// is seen by an interval of tokens.  A block without any takes the path without masks.
// A unit, as the writer describes it to all warps.
struct __align__(16) WTileUnit {
  int b, hk, k0, k1;   // keys [k0, k1) of a sequence and K/V head
  int len, fresh, lo;  // the sequence's tokens, new ones, first key whose weight changes
  int last;            // no unit: the ones before were all
  int ta, tb;          // tokens that see some of the keys
  int ca, cb;          // tokens that see all of them
};
static_assert(sizeof(WTileUnit) == 48, "three 16-byte words");

template <int D>
struct WTileCfg {
  static constexpr int kThreads = 640, kWarpProd = 16, kWarpMma = 17, kWarpSide = 18;
  static constexpr int kUnit = 2 * kWeightTile;          // keys
  static constexpr int kBoxes = D / 64;
  static constexpr uint32_t kBox = 128u * 128u;
  static constexpr uint32_t kTileBytes = kBoxes * kBox;  // 128 rows of K or Q
  static constexpr int kRing = D == 128 ? 6 : 8;
  static constexpr int kPiece = 32;                      // rows of a box of Q
  static constexpr uint32_t kSideBytes = 2 * 512 + 16;   // -L and token of 128 rows; their number, negative: masks wanted
  static constexpr uint32_t kSideOff = kRing * kTileBytes;
  static constexpr int kMaxCluster = 4;
  static constexpr uint32_t kSumBytes = kUnit * 4;
  static constexpr uint32_t kJoinOff = kSideOff + 2 * kSideBytes;  // [2 units] sums of two groups, of each other CTA
  static constexpr uint32_t kJoinBytes = (2 + kMaxCluster - 1) * kSumBytes;
  static constexpr int kUnits = 8;  // descriptions of units
  static constexpr uint32_t kUnitOff = kJoinOff + 2 * kJoinBytes;
  static constexpr uint32_t kBarOff = kUnitOff + kUnits * sizeof(WTileUnit);
  static constexpr uint32_t kTmemSlot = kBarOff + (16 + 2 * kRing + 2 * kUnits + 1) * 8;
  static constexpr uint32_t kAbort = kTmemSlot + 4;
  static constexpr uint32_t kSmemBytes = kAbort + 4;
  static constexpr uint32_t kTmemCols = 512;
  static_assert(kBarOff % 8 == 0 && kSideBytes % 16 == 0 && kUnitOff % 16 == 0, "alignment");
  static_assert(kSmemBytes <= 232448, "shared memory budget");
};

__device__ __forceinline__ void tma_prefetch_4d(const CUtensorMap* map, int x, int y, int z, int w) {
  asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %2, %3, %4}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}
// `bytes` (a multiple of 16) of this CTA's shared memory into another's, counted by a barrier there.
__device__ __forceinline__ void copy_to_cta(uint32_t dst, uint32_t src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "r"(src), "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// One arrival for the whole warp.
__device__ __forceinline__ void mbar_arrive_warp(uint32_t bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

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

// The tokens [ta, tb) that see key `key`.
__device__ __forceinline__ void key_tokens(const WeightsParams& p, int len, int fresh, int key, int& ta, int& tb) {
  const long long base = static_cast<long long>(len) - fresh;
  long long a = 0, b = fresh;
  if (p.s.right >= 0) a = max(a, key - base - p.s.right);
  if (p.s.left >= 0) b = min(b, key - base + p.s.left + 1);
  ta = static_cast<int>(min(a, static_cast<long long>(fresh)));
  tb = static_cast<int>(max(b, 0ll));
}

// The units of a cluster, in a whole converged warp that describes 32 at a time, one to a lane.  Short units: its
// number and every (number of clusters)-th after it.  Long ones differ by whole sequences' row blocks, and a cluster has
// few of them, so each goes to the cluster that has least to do so far; every cluster finds the same assignment for
// itself, beside the products of its units (about 0.09 us for each unit of the call).  32/8 heads of 128, us so / in turn:
// 2 x up to 2048 tokens over 8192 115 / 132, another two 141 / 149, prompts of 4 x up to 4096 (64 heads) 279 / 348, one of
// 8192 271 / 324; where units are shorter, 4 x up to 1024 over 8192 141 / 132, 8 x up to 512 over 4096 132 / 89.
struct WTileUnits {
  static constexpr int kMost = 3;  // clusters of a lane: 96 of a launch
  WTileUnit mine;      // of this lane
  long long u;         // its number
  int b_from;          // sequences before it are behind all units to come
  long long first;     // first unit of that one
  int at;              // lane of the next unit
  int cluster, clusters;
  bool uneven;
  unsigned cost;         // of this lane's unit
  unsigned load[kMost];  // of clusters lane, lane + 32, ...: blocks, and the number in the low 8 bits
  __device__ __forceinline__ void copy(WTileUnit& v, int lane) const {
    const int* const from = reinterpret_cast<const int*>(&mine);
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(WTileUnit) / 4); ++i)
      reinterpret_cast<int*>(&v)[i] = __shfl_sync(0xffffffffu, from[i], lane);
  }
  // What this lane's unit keeps a CTA busy for, in row blocks above the cluster's number (its ends count for two); 0: none.
  __device__ __forceinline__ void weigh(const WeightsParams& p) {
    const int blocks = mine.tb <= mine.ta ? 0
                       : p.s.T >= 128     ? (mine.tb - mine.ta + 127) / 128 * p.group
                                          : (p.s.rows + 127) / 128;
    const int ranks = static_cast<int>(cluster_size());
    const int each = ranks == 1 ? blocks : (ranks == 2 ? (blocks + 1) >> 1 : (blocks + 3) >> 2);
    cost = mine.last ? 0u : static_cast<unsigned>(min(each, 1 << 14) + 2) << 8;
  }
  // Whether units keep a CTA busy for 20 row blocks and more on average (17 us; the search for one 7 us).
  __device__ __forceinline__ bool long_units(const WeightsParams& p) const {
    long long more = 0;
    for (int b = threadIdx.x & 31; b < p.s.B; b += 32) {
      const SeqKeys s = weight_keys(p, b);
      const long long each = static_cast<long long>((s.fresh + 127) / 128) * p.group - 20 * cluster_size();
      more += (tiles_of(s.lo, s.hi, kWeightTile) + 1) / 2 * each;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) more += __shfl_xor_sync(0xffffffffu, more, o);
    return more >= 0;
  }
  // The first unit into v.
  __device__ __forceinline__ void begin(const WeightsParams& p, WTileUnit& v) {
    const int lane = threadIdx.x & 31;
    uneven = p.uneven && long_units(p);
    cluster = static_cast<int>(blockIdx.x / cluster_size());
    clusters = static_cast<int>(gridDim.x / cluster_size());
    mine = {};  // the description that there is no unit has no row blocks either, whoever walks over them
    b_from = 0;
    first = 0;
    if (!uneven) {
      u = cluster + static_cast<long long>(lane) * clusters;
      fill(p);
      copy(v, 0);
      at = 1;
      return;
    }
    // nobody has anything to do: unit i goes to cluster i
#pragma unroll
    for (int r = 0; r < kMost; ++r) {
      const int c = 32 * r + lane;
      load[r] = 0xffffffffu;
      if (32 * r >= clusters) continue;
      u = min(c, clusters - 1);
      fill(p);
      weigh(p);
      if (c < clusters) load[r] = cost | static_cast<unsigned>(c);
      if (cluster / 32 == r) copy(v, cluster % 32);
    }
    u = clusters + lane - 32;
    at = 32;
  }
  // The next one into v.
  __device__ __forceinline__ void next(const WeightsParams& p, WTileUnit& v) {
    for (;;) {
      if (at == 32) {
        u += uneven ? 32 : 32ll * clusters;
        fill(p);
        at = 0;
        if (uneven) {  // only differences count
          weigh(p);
          unsigned least = 0xffffffffu;
#pragma unroll
          for (int r = 0; r < kMost; ++r) least = min(least, load[r]);
          least = __reduce_min_sync(0xffffffffu, least) & ~0xffu;
#pragma unroll
          for (int r = 0; r < kMost; ++r)
            if (load[r] != 0xffffffffu) load[r] -= least;
        }
      }
      const int j = at++;
      const unsigned more = uneven ? __shfl_sync(0xffffffffu, cost, j) : 0u;
      if (more == 0) {
        copy(v, j);
        return;
      }
      unsigned least = 0xffffffffu;
#pragma unroll
      for (int r = 0; r < kMost; ++r) least = min(least, load[r]);
      least = __reduce_min_sync(0xffffffffu, least);
#pragma unroll
      for (int r = 0; r < kMost; ++r)
        if (load[r] == least) load[r] += more;
      if (static_cast<int>(least & 0xffu) == cluster) {
        copy(v, j);
        return;
      }
    }
  }
  __device__ __forceinline__ void fill(const WeightsParams& p) {
    const int lane = threadIdx.x & 31;
    mine.last = 1;
    while (b_from < p.s.B) {
      SeqKeys s = {};
      int n = 0;
      if (b_from + lane < p.s.B) {
        s = weight_keys(p, b_from + lane);
        n = (tiles_of(s.lo, s.hi, kWeightTile) + 1) / 2;
      }
      long long incl = static_cast<long long>(p.s.Hk) * n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
      }
      // the first of the 32 sequences that ends behind this lane's unit
      int j = 0;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        if (u - first >= __shfl_sync(0xffffffffu, incl, j + o - 1)) j += o;
      const long long all = __shfl_sync(0xffffffffu, incl, 31);
      const bool here = mine.last && u - first < all;
      const long long before = __shfl_sync(0xffffffffu, incl, max(j - 1, 0));
      const int sn = __shfl_sync(0xffffffffu, n, j), len = __shfl_sync(0xffffffffu, s.len, j),
                fresh = __shfl_sync(0xffffffffu, s.fresh, j), lo = __shfl_sync(0xffffffffu, s.lo, j),
                hi = __shfl_sync(0xffffffffu, s.hi, j);
      if (here) {
        const long long in = u - first - (j > 0 ? before : 0);
        mine.last = 0;
        mine.b = b_from + j;
        mine.hk = static_cast<int>(quotient(in, sn));
        mine.k0 = (lo / kWeightTile + 2 * static_cast<int>(in - static_cast<long long>(mine.hk) * sn)) * kWeightTile;
        mine.k1 = min(mine.k0 + 2 * kWeightTile, hi);
        mine.len = len;
        mine.fresh = fresh;
        mine.lo = lo;
        key_tokens(p, len, fresh, mine.k0, mine.ta, mine.cb);  // the first key's tokens begin and end first
        key_tokens(p, len, fresh, mine.k1 - 1, mine.ca, mine.tb);
      }
      if (!__any_sync(0xffffffffu, mine.last)) return;
      b_from += 32;
      first += all;
    }
  }
};

// The row blocks of a unit that this CTA takes, every (CTAs of the cluster)-th.  With 128 tokens or more a block
// holds tokens of one query head, of those that see some key of the unit; with fewer it holds rows of several heads,
// whatever they see.  Found by additions alone: each role walks over the blocks for itself, with a few hundred cycles for
// one.
struct WTileBlocks {
  int head, part, left;  // query head of the group (0: blocks over all rows), block in its tokens, blocks to come
  int per;               // blocks of a head
  int first, end;        // rows (of a head) that the blocks cover
  int rank, ranks;       // this CTA in its cluster
  __device__ __forceinline__ WTileBlocks(const WeightsParams& p, const WTileUnit& w)
      : rank(static_cast<int>(cluster_rank())), ranks(static_cast<int>(cluster_size())) {
    const bool single = p.s.T >= 128;
    first = single ? w.ta : 0;
    end = single ? w.tb : p.s.rows;
    per = w.tb > w.ta ? (end - first + 127) / 128 : 0;
    left = per * (single ? p.group : 1) - rank;
    head = 0;
    part = rank;
    wrap();
  }
  __device__ __forceinline__ void wrap() {
    if (left > 0)
      while (part >= per) {
        part -= per;
        ++head;
      }
  }
  __device__ __forceinline__ explicit operator bool() const { return left > 0; }
  __device__ __forceinline__ void step() {
    left -= ranks;
    part += ranks;
    wrap();
  }
  __device__ __forceinline__ int count() const { return left > 0 ? (left - 1) / ranks + 1 : 0; }
  __device__ __forceinline__ int row(const WeightsParams& p) const { return head * p.s.T + first + part * 128; }
  __device__ __forceinline__ int rows() const { return min(128, end - first - part * 128); }
  // some row does not see all keys of the unit (its LSE aside), or the columns of 32 hold more than the rows
  __device__ __forceinline__ bool cut(const WeightsParams& p, const WTileUnit& w) const {
    const int n = rows(), t = first + part * 128;
    if (n & 31) return true;
    return p.s.T >= 128 ? t < w.ca || t + n > w.cb : w.ca > 0 || w.cb < p.s.T;
  }
};

template <int D>
__global__ void __launch_bounds__(WTileCfg<D>::kThreads, 1)
    fa_kv_weights_tile_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmQ,
                              const WeightsParams p) {
  using C = WTileCfg<D>;
  extern __shared__ __align__(1024) uint8_t wtile_smem[];
  const uint32_t base = smem_addr(wtile_smem);  // 1024-byte aligned: the kernel has no static shared memory
  const uint32_t bar0 = base + C::kBarOff;
  auto bar = [&](int i) -> uint32_t { return bar0 + 8u * static_cast<uint32_t>(i); };
  auto s_full = [&](int buf, int tile) -> uint32_t { return bar(2 * buf + tile); };  // S and its side buffer written
  auto s_free = [&](int buf, int tile) -> uint32_t { return bar(4 + 2 * buf + tile); };  // both read
  auto sums_full = [&](int slot) -> uint32_t { return bar(8 + slot); };   // the groups' sums of a unit
  auto sums_free = [&](int slot) -> uint32_t { return bar(10 + slot); };
  auto join_full = [&](int slot) -> uint32_t { return bar(12 + slot); };  // the other CTAs' (first CTA)
  auto join_free = [&](int slot) -> uint32_t { return bar(14 + slot); };  // (other CTAs)
  auto full = [&](int i) -> uint32_t { return bar(16 + i); };
  auto empty = [&](int i) -> uint32_t { return bar(16 + C::kRing + i); };
  auto unit_full = [&](int i) -> uint32_t { return bar(16 + 2 * C::kRing + i); };  // a unit described
  auto unit_free = [&](int i) -> uint32_t { return bar(16 + 2 * C::kRing + C::kUnits + i); };
  const uint32_t drain = bar(16 + 2 * C::kRing + 2 * C::kUnits);
  WTileUnit* const units = reinterpret_cast<WTileUnit*>(wtile_smem + C::kUnitOff);
  const int rank = static_cast<int>(cluster_rank()), ranks = static_cast<int>(cluster_size());
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
      for (int tile = 0; tile < 2; ++tile) {
        mbar_init(s_full(i, tile), 2);
        mbar_init(s_free(i, tile), 4);
      }
      mbar_init(sums_full(i), 16);
      mbar_init(sums_free(i), 1);
      mbar_init(join_full(i), 1);
      mbar_init(join_free(i), 1);
    }
    for (int i = 0; i < C::kRing; ++i) {
      mbar_init(full(i), 1);
      mbar_init(empty(i), 1);
    }
    for (int i = 0; i < C::kUnits; ++i) {
      mbar_init(unit_full(i), 1);
      mbar_init(unit_free(i), C::kThreads / 32);
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
  if (warp == C::kWarpMma) {
    tmem_alloc(smem_addr(tmem_slot), C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncwarp();
  cluster_sync();  // and the barriers of all CTAs are there
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int rows = p.s.rows;
  WTileUnit w = {};
  int units_read = 0;
  bool ok = true;
  // the next unit as the writer described it; false: none, or a wait gave up
  auto read_unit = [&](WTileUnit& v) -> bool {
    const int i = units_read % C::kUnits;
    ok = uniform(mbar_wait(unit_full(i), (units_read / C::kUnits) & 1, abort_flag));
    if (!ok) return false;
    ++units_read;
    v = units[i];
    mbar_arrive_warp(unit_free(i));
    return !v.last;
  };
  auto next_unit = [&]() -> bool { return read_unit(w); };

  if (warp == C::kWarpProd) {
    // ======================= TMA producer =================================
    const int chunk = min(1 << p.s.page_shift, kWeightTile);  // keys of one box
    const int piece = lane / C::kBoxes, x = lane % C::kBoxes;
    WSlots slots(C::kRing);
    uint32_t used = 0;  // slots with a copy in flight or landed
    auto take = [&]() -> int {  // the next slot, once it is free
      uint32_t parity;
      const int s = slots.take(parity);
      ok = uniform(mbar_wait(empty(s), parity ^ 1u, abort_flag));
      if (!ok) slots.phase ^= 1u << s;  // no copy was issued
      else used |= 1u << s;
      return s;
    };
    // this lane's box of a tile of a unit's keys: its first key, and whether it is wanted
    auto key_of = [&](const WTileUnit& v, int tile) -> int { return v.k0 + tile * kWeightTile + piece * chunk; };
    auto wanted = [&](const WTileUnit& v, int tile) -> bool {
      const int key = key_of(v, tile);
      return lane < kWeightTile / chunk * C::kBoxes && key < v.k1 && key + chunk > v.lo;
    };
    auto page_of = [&](const WTileUnit& v, int tile) -> int {
      return wanted(v, tile)
                 ? coherent(p.s.table + static_cast<long long>(v.b) * p.s.max_pages + (key_of(v, tile) >> p.s.page_shift))
                 : -1;
    };
    int page[2] = {-1, -1};
    if (next_unit()) {
      page[0] = page_of(w, 0);
      page[1] = page_of(w, 1);
    }
    while (ok && !w.last) {
      // the next unit's pages are read, and its K brought to L2, while this one's row blocks are loaded; where finding it
      // takes long, not before some of them
      WTileUnit v;
      int next_page[2] = {-1, -1}, wait = p.uneven ? min(8, max(WTileBlocks(p, w).count() - 1, 0)) : 0;
      auto look = [&]() {
        if (!read_unit(v)) return;
        next_page[0] = page_of(v, 0);
        next_page[1] = page_of(v, 1);
#pragma unroll
        for (int tile = 0; tile < 2; ++tile)
          if (static_cast<unsigned>(next_page[tile]) < static_cast<unsigned>(p.s.n_pages))
            tma_prefetch_4d(&tmK, x * 64, key_of(v, tile) & ((1 << p.s.page_shift) - 1), v.hk, next_page[tile]);
      };
      int k_slot[2] = {-1, -1};
      for (WTileBlocks at(p, w); at; at.step()) {
        if (k_slot[0] < 0) {
#pragma unroll
          for (int tile = 0; tile < 2; ++tile) {
            if (!ok || w.k0 + tile * kWeightTile >= w.k1) continue;
            const bool load = wanted(w, tile);
            if (load && static_cast<unsigned>(page[tile]) >= static_cast<unsigned>(p.s.n_pages))
              atomicOr(p.s.status, kPagedPage);
            const unsigned boxes = __popc(__ballot_sync(0xffffffffu, load));
            const int s = k_slot[tile] = take();
            if (!ok) continue;
            if (lane == 0) mbar_arrive_expect_tx(full(s), boxes * chunk * 128u);
            __syncwarp();
            if (load)
              tma_load_4d(base + s * C::kTileBytes + x * C::kBox + piece * chunk * 128, &tmK, full(s), x * 64,
                          key_of(w, tile) & ((1 << p.s.page_shift) - 1), w.hk, page[tile]);
          }
          if (!ok) break;
        }
        if (wait-- == 0) look();
        if (!ok) break;
        const int s = take();
        if (!ok) break;
        const int pieces = (at.rows() + C::kPiece - 1) / C::kPiece;
        if (lane == 0) mbar_arrive_expect_tx(full(s), pieces * C::kBoxes * C::kPiece * 128u);
        __syncwarp();
        if (lane < pieces * C::kBoxes)
          tma_load_3d(base + s * C::kTileBytes + x * C::kBox + piece * C::kPiece * 128, &tmQ, full(s), x * 64,
                      static_cast<int>((static_cast<long long>(w.b) * p.s.Hk + w.hk) * rows) + at.row(p) + piece * C::kPiece, 0);
        slots.give(s);
      }
#pragma unroll
      for (int tile = 0; tile < 2; ++tile)
        if (k_slot[tile] >= 0) slots.give(k_slot[tile]);
      if (ok && wait >= 0) look();
      w = v;
      page[0] = next_page[0];
      page[1] = next_page[1];
    }
    if (!ok) failed(2u);
    if (*abort_flag) {  // let every copy issued land before the CTA's shared memory goes
      for (int s = 0; s < C::kRing; ++s)
        if ((used >> s) & 1u) uniform(mbar_wait(full(s), ((slots.phase >> s) & 1u) ^ 1u, nullptr));
    }
  } else if (warp == C::kWarpMma) {
    // ======================= MMA issuer ===================================
    // Descriptors differ in their low words alone (the address), so those are kept, and every index is a constant: with
    // arrays indexed at run time an MMA took 100 cycles and more to issue, 64 to run.
    const uint64_t ring = sdesc_sw128(base, 16, 1024);
    const uint32_t ring_lo = static_cast<uint32_t>(ring), ring_hi = static_cast<uint32_t>(ring >> 32);
    auto desc = [&](uint32_t lo) -> uint64_t { return (static_cast<uint64_t>(ring_hi) << 32) | lo; };
    WSlots slots(C::kRing);
    int block = 0;
    auto take = [&]() -> int {  // the next tile's slot, once it has landed
      uint32_t parity;
      const int s = slots.take(parity);
      ok = uniform(mbar_wait(full(s), parity, abort_flag));
      return s;
    };
    auto low = [&](int slot) -> uint32_t { return ring_lo + ((slot * C::kTileBytes) >> 4); };
    while (next_unit()) {
      int k_slot0 = -1, k_slot1 = -1;
      uint32_t k0 = 0, k1 = 0;
      const bool two = w.k0 + kWeightTile < w.k1;
      for (WTileBlocks at(p, w); at; at.step()) {
        if (k_slot0 < 0) {
          k_slot0 = take();
          if (ok && two) k_slot1 = take();
          if (!ok) break;
          k0 = low(k_slot0);
          k1 = low(k_slot1);
        }
        const int q_slot = take();
        if (!ok) break;
        const uint32_t q = low(q_slot), buf = block & 1, ph = ((block >> 1) & 1) ^ 1u;
        const uint32_t idesc = idesc_bf16(128, (at.rows() + 31) & ~31, false);
        auto scores = [&](uint32_t k, uint32_t dst) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = ((kk >> 2) * C::kBox + (kk & 3) * 32) >> 4;
            mma_ss_elect(dst, desc(k + off), desc(q + off), idesc, kk > 0 ? 1u : 0u);
          }
        };
        ok = uniform(mbar_wait(s_free(buf, 0), ph, abort_flag));
        if (!ok) break;
        tc_fence_after();
        scores(k0, tmem + buf * 256);
        mma_commit_elect(s_full(buf, 0));
        ok = uniform(mbar_wait(s_free(buf, 1), ph, abort_flag));
        if (!ok) break;
        tc_fence_after();
        if (two) scores(k1, tmem + buf * 256 + 128);
        mma_commit_elect(empty(q_slot));
        mma_commit_elect(s_full(buf, 1));
        slots.give(q_slot);
        ++block;
      }
      if (!ok) break;
      if (k_slot0 >= 0) {
        mma_commit_elect(empty(k_slot0));
        slots.give(k_slot0);
      }
      if (k_slot1 >= 0) {
        mma_commit_elect(empty(k_slot1));
        slots.give(k_slot1);
      }
    }
    if (!ok) failed(4u);
    mma_commit_elect(drain);
    uniform(mbar_wait(drain, 0, nullptr));
  } else if (warp == C::kWarpSide) {
    // ======================= LSE and tokens of the rows ====================
    // A block is handed over before the next one is looked for: units without blocks may lie between, more of them than
    // the writer describes ahead of this block's unit, whose sums wait for it.
    int block = 0;
    bool more = next_unit();
    WTileBlocks at(p, w);
    float l2[4];  // LSE of the block's rows, on their way while the S buffer is waited for
    auto seek = [&]() {
      while (more && !at) {
        more = next_unit();
        if (more) at = WTileBlocks(p, w);
      }
      if (!more) return;
      const float* const lse = p.s.lse + (static_cast<long long>(w.b) * p.s.Hk + w.hk) * rows + at.row(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) l2[i] = 32 * i + lane < at.rows() ? lse[32 * i + lane] : 0.f;
    };
    if (more) seek();
    while (more) {
      const int n = at.rows(), buf = block & 1;
      int t[4];
      bool cut = at.cut(p, w);
      const int t0 = p.s.T >= 128 ? at.first + at.part * 128 : 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 32 * i + lane;
        t[i] = t0 + r;
        if (p.s.T < 128) t[i] = at.row(p) + r - row_head(p, at.row(p) + r) * p.s.T;
        if (r >= n) t[i] = 0x7fffffff;
      }
      float l[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (l2[i] == -__int_as_float(0x7f800000)) {  // a row without a key
          t[i] = 0x7fffffff;
          cut = true;
        }
        l[i] = l2[i] * -1.44269504f;
      }
      cut = !uniform(!cut);
      const uint32_t ph = ((block >> 1) & 1) ^ 1u;
      ok = ok && uniform(mbar_wait(s_free(buf, 0), ph, abort_flag) && mbar_wait(s_free(buf, 1), ph, abort_flag));
      if (!ok) break;
      uint8_t* const side = wtile_smem + C::kSideOff + buf * C::kSideBytes;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        reinterpret_cast<float*>(side)[32 * i + lane] = l[i];
        reinterpret_cast<int*>(side + 512)[32 * i + lane] = t[i];
      }
      if (lane == 0) *reinterpret_cast<int*>(side + 1024) = cut ? -n : n;
      mbar_arrive_warp(s_full(buf, 0));
      mbar_arrive_warp(s_full(buf, 1));
      ++block;
      at.step();
      seek();
    }
    if (!ok) failed(32u);
  } else if (warp > C::kWarpSide) {
    // ======================= writer, planner ===============================
    WTileUnits list;
    WTileUnit plan;
    int told = 0;
    auto tell = [&]() {  // one more unit, described to all warps; the last one says that there is none
      if (told == 0) list.begin(p, plan);
      else if (!plan.last) list.next(p, plan);
      else return;
      const int i = told % C::kUnits;
      ok = uniform(mbar_wait(unit_free(i), ((told / C::kUnits) & 1) ^ 1u, abort_flag));
      if (!ok) return;
      if (lane == 0) units[i] = plan;
      mbar_arrive_warp(unit_full(i));
      ++told;
    };
    // so many before the first sums are waited for: where finding one takes long, only as many as the rest needs
    tell();
    for (int i = list.uneven ? 2 : C::kUnits - 2; i > 0 && ok; --i) tell();
    int unit = 0;
    while (ok && next_unit()) {
      float* to[8];
      float old[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int key = w.k0 + 32 * i + lane;
        to[i] = nullptr;
        old[i] = 0.f;
        if (rank == 0 && key >= w.lo && key < w.k1) {
          const int page = coherent(p.s.table + static_cast<long long>(w.b) * p.s.max_pages + (key >> p.s.page_shift));
          if (static_cast<unsigned>(page) < static_cast<unsigned>(p.s.n_pages)) {
            to[i] = p.w + page * p.w_page + w.hk * p.w_head + (key & ((1 << p.s.page_shift) - 1));
            if (p.decay != 0.f && key < w.len - w.fresh) old[i] = p.decay * *to[i];
          } else {
            atomicOr(p.s.status, kPagedPage);
          }
        }
      }
      const int slot = unit & 1;
      const uint32_t ph = (unit >> 1) & 1;
      ++unit;
      float* const sums = reinterpret_cast<float*>(wtile_smem + C::kJoinOff + slot * C::kJoinBytes) + lane;
      ok = uniform(mbar_wait(sums_full(slot), ph, abort_flag));
      if (!ok) break;
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = sums[32 * i] + sums[C::kUnit + 32 * i];
      if (rank != 0) {
        // the joined sums lie where the first group's were until the first CTA has them
#pragma unroll
        for (int i = 0; i < 8; ++i) sums[32 * i] = v[i];
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0)
          copy_to_cta(in_cta(base + C::kJoinOff + slot * C::kJoinBytes + (1 + rank) * C::kSumBytes, 0),
                      base + C::kJoinOff + slot * C::kJoinBytes, C::kSumBytes, in_cta(join_full(slot), 0));
        ok = uniform(mbar_wait(join_free(slot), ph, abort_flag));
        if (!ok) break;
      } else if (ranks > 1) {
        if (lane == 0) mbar_arrive_expect_tx(join_full(slot), (ranks - 1) * C::kSumBytes);
        ok = uniform(mbar_wait(join_full(slot), ph, abort_flag));
        if (!ok) break;
        for (int r = 1; r < ranks; ++r)
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] += sums[(1 + r) * C::kUnit + 32 * i];
        __syncwarp();
        if (lane > 0 && lane < ranks) mbar_arrive_cluster(in_cta(join_free(slot), lane));
      }
      mbar_arrive_warp(sums_free(slot));
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (to[i]) *to[i] = old[i] + v[i];
      tell();
    }
    if (!ok) failed(8u);
  } else {
    // ======================= exponentials and sums =========================
    const int buf = warp >> 3, tile = (warp >> 2) & 1, quarter = warp & 3;
    const uint32_t lanes = tmem + (2 * buf + tile) * 128 + (static_cast<uint32_t>(quarter * 32) << 16);
    float* const sums = reinterpret_cast<float*>(wtile_smem + C::kJoinOff) + buf * C::kUnit + tile * kWeightTile +
                        quarter * 32 + lane;
    const uint8_t* const side = wtile_smem + C::kSideOff + buf * C::kSideBytes;
    const float c = p.s.scale_log2;
    int block = 0, unit = 0;  // blocks of the units before, units before
    uint32_t phase = 0;       // of this group's blocks
    float sum[4];
    // rows g .. g + 15 of a block, one key
    auto add = [&](auto masks, const uint32_t(&r)[16], int g, int ta, int tb) {
      const float4* const l4 = reinterpret_cast<const float4*>(side) + g / 4;
      const int4* const t4 = reinterpret_cast<const int4*>(side + 512) + g / 4;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 l = l4[i];
        float x0, x1, x2, x3;
        fma2c(x0, x1, __uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1]), c, l.x, l.y);
        fma2c(x2, x3, __uint_as_float(r[4 * i + 2]), __uint_as_float(r[4 * i + 3]), c, l.z, l.w);
        x0 = ex2(x0);
        x1 = ex2(x1);
        x2 = ex2(x2);
        x3 = ex2(x3);
        if constexpr (decltype(masks)::value) {
          const int4 t = t4[i];
          x0 = t.x >= ta && t.x < tb ? x0 : 0.f;
          x1 = t.y >= ta && t.y < tb ? x1 : 0.f;
          x2 = t.z >= ta && t.z < tb ? x2 : 0.f;
          x3 = t.w >= ta && t.w < tb ? x3 : 0.f;
        }
        add2(sum[0], sum[1], x0, x1);
        add2(sum[2], sum[3], x2, x3);
      }
    };
    // a block's n rows: 16 columns are loaded while the 16 before them are worked on
    auto add_block = [&](auto masks, int n, int ta, int tb) {
      uint32_t ra[16], rb[16];
      tmem_ld16(lanes, ra);
      tmem_ld_wait16(ra);
#pragma unroll 1
      for (int g = 0; g < n; g += 32) {
        tmem_ld16(lanes + g + 16, rb);
        add(masks, ra, g, ta, tb);
        tmem_ld_wait16(rb);
        if (g + 32 < n) tmem_ld16(lanes + g + 32, ra);
        add(masks, rb, g + 16, ta, tb);
        if (g + 32 < n) tmem_ld_wait16(ra);
      }
    };
    while (next_unit()) {
      const int key = w.k0 + tile * kWeightTile + quarter * 32 + lane;
      const bool some = w.k0 + tile * kWeightTile < w.k1;  // the tile has keys
      int ta, tb;
      key_tokens(p, w.len, w.fresh, key, ta, tb);
      sum[0] = sum[1] = sum[2] = sum[3] = 0.f;
      const int blocks = WTileBlocks(p, w).count();
      for (int i = (block ^ buf) & 1; i < blocks; i += 2) {
        ok = uniform(mbar_wait(s_full(buf, tile), phase, abort_flag));
        if (!ok) break;
        phase ^= 1u;
        tc_fence_after();
        if (some) {
          const int n = *reinterpret_cast<const int*>(side + 1024);
          if (n < 0) add_block(std::true_type{}, -n, ta, tb);
          else add_block(std::false_type{}, n, ta, tb);
        }
        tc_fence_before();
        mbar_arrive_warp(s_free(buf, tile));
      }
      block += blocks;
      if (!ok) break;
      const int slot = unit & 1;
      ok = uniform(mbar_wait(sums_free(slot), ((unit >> 1) & 1) ^ 1u, abort_flag));
      if (!ok) break;
      ++unit;
      sums[slot * (C::kJoinBytes / 4)] = (sum[0] + sum[1]) + (sum[2] + sum[3]);
      mbar_arrive_warp(sums_full(slot));
    }
    if (!ok) failed(1u);
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();  // nothing of another CTA is on its way here
  if (warp == C::kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

}  // namespace fa
