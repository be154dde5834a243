// fa_paged_tile.cuh -- paged attention for many query rows per K/V head, on the
// tcgen05 path: the shared prefix (its row blocks run over the batch) and
// sequences with more rows than the warp-level kernel takes.
//
// One persistent CTA per SM streams its share of 128-key tiles past its row
// blocks: S = Q K^T and O += P V as tcgen05 MMAs with S, P and O in TMEM, K and V
// boxes by TMA straight from the pages, softmax in two warpgroups that work
// while the other one's products run.  What the two warpgroups share out:
//   PAIR (row blocks of 256): warpgroup t owns query tile t of 128 rows and
//     meets every key tile, as in fa_fwd_kernel, so each K/V byte is read from
//     L2 once per 256 rows;
//   else (row blocks of 128): warpgroup t owns the key tiles t, t + 2, ... of the
//     one query tile, with its own O in TMEM; the two are joined at the end of
//     the row block.
//   warps 0-3, 4-7  softmax, correction, epilogue (thread = row = TMEM lane)
//   warp 8          TMA producer: K and V tiles in the order the MMAs take them,
//                   one lane per page box
//   warp 9          MMA issuer
//   warps 10-11     load the rows of Q of the segment ahead into swizzled
//                   shared memory
// A segment's end (epilogue) overlaps the next one's Q load, K/V loads and first
// scores.  TMEM (512 columns): S0 [0, 128), S1 [128, 256), O0, O1 from 256; P (bf16)
// overwrites the first 64 columns of its S.
// Keys outside the segment's range (the end of a page, pages given back below a
// window) are masked in S; their V rows, which may hold anything, are zeroed in
// shared memory by the softmax warps before they hand over P (0 * NaN is NaN).
//
// Bound: with few rows DRAM (a tile's K and V, 64 KB at D = 128, take 1.5 us of an
// SM's share of 6.8 TB/s; loop alone about 7 TB/s on 32 rows), with a pair the
// tensor pipe (1.5 us a tile against 1.35 at the measured bf16 rate; 2 x 256
// tokens of 32/8 heads over 65536 keys: 1270-1360 TFLOP/s).  Short calls are bound
// by what the loop does not cover: 6 us to the first scores (the lengths, then
// 224 KB of Q, K and V per SM at once), 3 us for the last row block's output, the
// merge.
#pragma once

#include "fa_paged_kernel.cuh"

namespace fa {

template <int D, bool PAIR>
struct TileCfg {
  static constexpr int kRows = PAIR ? 256 : 128, kTile = kPagedTile;
  static constexpr int kThreads = 384, kWarpProd = 8, kWarpMma = 9;
  static constexpr int kBoxes = D / 64;
  static constexpr uint32_t kBox = 128u * 128u;
  static constexpr uint32_t kTileBytes = kBoxes * kBox;  // 128 rows of Q, K or V
  static constexpr int kRing = D == 128 ? 5 : 8;
  static constexpr uint32_t kRingOff = 2 * kTileBytes;   // after two Q tiles (PAIR) or Q buffers
  static constexpr uint32_t kStatOff = kRingOff + kRing * kTileBytes;  // [2 warpgroups][128] (L, 1 / l)
  static constexpr uint32_t kBarOff = kStatOff + (PAIR ? 0 : 2 * 128 * 8);
  static constexpr uint32_t kSmemBytes = kBarOff + 1024;
  static constexpr uint32_t kTmemCols = 512, kTmO = 256;
  static constexpr uint32_t kIdescS = idesc_bf16(128, 128, false);
  static constexpr uint32_t kIdescO = idesc_bf16(128, D, true);
  // registers per thread: at launch (checked by the host), softmax warpgroups, warpgroup 2
  static constexpr int kRegLaunch = 168, kRegSoftmax = D == 64 ? 192 : 184, kRegMisc = D == 64 ? 120 : 128;
  static_assert(2 * 128 * kRegSoftmax + 128 * kRegMisc <= kThreads * kRegLaunch, "register split");
  static_assert(kSmemBytes <= 232448, "shared memory budget");
};

// barrier slots (8 bytes each); the rest of the 512-byte block: scratch of
// paged_share at 256, TMEM base at 448, abort flag at 452
enum : int {
  kTBarQ = 0,      // [2] Q tile or buffer loaded
  kTBarQFree = 2,  // [2] no score product reads it any more
  kTBarS = 4,      // [2]
  kTBarP = 6,      // [2]
  kTBarFinal = 8,  // [2] the segment's last product is complete (PAIR: of each query tile)
  kTBarStat = 10,  // both warpgroups' row statistics are in shared memory
  kTBarEpi = 11,   // the epilogue has read O
  kTBarDrain = 12,
  kTBarRing = 13   // full[kRing] then empty[kRing]
};
constexpr uint32_t kTileScratchOff = 256, kTileTmemOff = 448, kTileAbortOff = 452;
constexpr uint32_t kTileWalkOff = 512;  // the softmax warps' walks, after the 512-byte block

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// The tiles [jlo, jhi) of the CTA's part that some row of the block sees.
template <int RB, int TILE, bool PREFIX>
__device__ __forceinline__ void seen_tiles(const PagedParams& p, const PagedWalk& w, int& jlo, int& jhi) {
  jlo = w.j;
  jhi = w.jend;
  if constexpr (!PREFIX) {
    const SeqKeys s = seq_keys(p, w.b);
    const int r0 = w.rb * RB, r1 = min(p.rows, r0 + RB) - 1;
    int t0 = 0, t1 = p.T - 1;  // tokens of the block's rows
    if (r0 / p.T == r1 / p.T) {
      t0 = r0 % p.T;
      t1 = r1 % p.T;
    }
    t1 = min(t1, s.fresh - 1);
    int lo = 0, hi = 0, unused;
    if (t0 <= t1) {
      row_own_keys(p, s, t0, lo, unused);
      row_own_keys(p, s, t1, unused, hi);
    }
    if (hi <= lo) {
      jhi = jlo;
      return;
    }
    jlo = max(jlo, lo / TILE - w.tile0);
    jhi = max(jlo, min(jhi, (hi + TILE - 1) / TILE - w.tile0));
  }
}

template <int D, bool PREFIX, bool PAIR>
__global__ void __launch_bounds__(TileCfg<D, PAIR>::kThreads, 1)
    fa_paged_tile_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                         const PagedParams p) {
  using C = TileCfg<D, PAIR>;
  using S = PagedSchedule<C::kRows, C::kTile, PREFIX>;
  extern __shared__ __align__(1024) uint8_t tile_smem[];
  const uint32_t base = smem_addr(tile_smem);  // 1024-byte aligned: the kernel has no static shared memory
  const uint32_t bar0 = base + C::kBarOff;
  auto bar = [&](int i) -> uint32_t { return bar0 + 8u * static_cast<uint32_t>(i); };
  auto full = [&](int slot) -> uint32_t { return bar(kTBarRing + slot); };
  auto empty = [&](int slot) -> uint32_t { return bar(kTBarRing + C::kRing + slot); };
  auto slot_addr = [&](int slot) -> uint32_t { return base + C::kRingOff + slot * C::kTileBytes; };
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(tile_smem + C::kBarOff + kTileTmemOff);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(tile_smem + C::kBarOff + kTileAbortOff);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto failed = [&](unsigned role) {
    *abort_flag = 1;
    atomicOr(p.status, kPagedTimeout | (role << 8));
  };
  auto uniform = [](bool v) -> bool { return __all_sync(0xffffffffu, v); };
  const bool beside = !PREFIX && p.prefix_len > 0;
  const int block = static_cast<int>(blockIdx.x);

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kTBarQ + i), 64);
      mbar_init(bar(kTBarQFree + i), 1);
      mbar_init(bar(kTBarS + i), 1);
      mbar_init(bar(kTBarP + i), 128);
      mbar_init(bar(kTBarFinal + i), 1);
    }
    mbar_init(bar(kTBarStat), 256);
    mbar_init(bar(kTBarEpi), 256);
    mbar_init(bar(kTBarDrain), 1);
    for (int i = 0; i < 2 * C::kRing; ++i) mbar_init(bar(kTBarRing + i), 1);
    *abort_flag = 0;
    mbar_init_fence();
    tma_prefetch_map(&tmK);
    tma_prefetch_map(&tmV);
  }
  paged_begin(beside);
  if (base & 1023u) {  // the swizzled layouts need it; the launch places it so
    if (threadIdx.x == 0) atomicOr(p.status, kPagedTimeout | (16u << 8));
    paged_end(beside);
    return;
  }
  PagedWalk w;
  bool first;  // the segment holds the share's first unit
  if (!paged_share<C::kRows, C::kTile, PREFIX, C::kThreads>(
          p, block, reinterpret_cast<long long*>(tile_smem + C::kBarOff + kTileScratchOff), w, first)) {
    paged_end(beside);
    return;
  }
  if (warp == C::kWarpMma) {
    tmem_alloc(smem_addr(tmem_slot), C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp >= 8) {
    regs_dec<C::kRegMisc>();
    if (warp == C::kWarpProd) {
      // ======================= TMA producer =================================
      const int chunk_rows = min(1 << p.page_shift, C::kTile);  // keys of one box: smaller pages take several
      const int piece = lane / C::kBoxes, x = lane % C::kBoxes;
      const bool mine = lane < C::kTile / chunk_rows * C::kBoxes;
      int item = 0;
      bool ok = true;
      do {
        int jlo, jhi;
        seen_tiles<C::kRows, C::kTile, PREFIX>(p, w, jlo, jhi);
        const int* const pages = S::pages(p, w);
        auto key_of = [&](int j) -> int { return (w.tile0 + j) * C::kTile + piece * chunk_rows; };
        auto wanted = [&](int k) -> bool { return mine && k < w.hi && k + chunk_rows > w.lo; };
        auto page_of = [&](int j) -> int {
          const int k = key_of(j);
          return (j < jhi && wanted(k)) ? coherent(pages + (k >> p.page_shift)) : -1;
        };
        auto put = [&](const CUtensorMap* map, int j, int page) -> bool {
          const int s = item % C::kRing;
          if (!uniform(mbar_wait(empty(s), ((item / C::kRing) & 1) ^ 1u, abort_flag))) return false;
          const int k = key_of(j);
          const bool load = wanted(k);
          const unsigned boxes = __popc(__ballot_sync(0xffffffffu, load));
          if (lane == 0) mbar_arrive_expect_tx(full(s), boxes * chunk_rows * 128u);
          __syncwarp();
          if (load) {
            if (map == &tmK && static_cast<unsigned>(page) >= static_cast<unsigned>(p.n_pages))
              atomicOr(p.status, kPagedPage);
            tma_load_4d(slot_addr(s) + x * C::kBox + piece * chunk_rows * 128, map, full(s), x * 64,
                        k & ((1 << p.page_shift) - 1), w.hk, page);
          }
          ++item;
          return true;
        };
        // page indices are read ahead of their use; each order is that of the MMA issuer
        int a = page_of(jlo), b = page_of(jlo + 1), c = page_of(jlo + 2);
        if constexpr (PAIR) {
          for (int j = jlo; ok && j < jhi; ++j) {
            const int d = page_of(j + 3);
            ok = put(&tmK, j, a) && put(&tmV, j, a);
            a = b;
            b = c;
            c = d;
          }
        } else {
          if (jlo < jhi) ok = put(&tmK, jlo, a) && (jlo + 1 >= jhi || put(&tmK, jlo + 1, b));
          for (int j = jlo; ok && j < jhi; ++j) {
            const int d = page_of(j + 3);
            ok = put(&tmV, j, a) && (j + 2 >= jhi || put(&tmK, j + 2, c));
            a = b;
            b = c;
            c = d;
          }
        }
      } while (ok && S::next(p, w));
      if (!ok) failed(2u);
      if (*abort_flag) {  // let every copy issued land before the CTA's shared memory goes
        for (int i = max(0, item - C::kRing); i < item; ++i)
          uniform(mbar_wait(full(i % C::kRing), (i / C::kRing) & 1, nullptr));
      }
    } else if (warp == C::kWarpMma) {
      // ======================= MMA issuer ===================================
      const uint64_t dQ = sdesc_sw128(base, 16, 1024);
      const uint64_t dK = sdesc_sw128(base + C::kRingOff, 16, 1024);
      const uint64_t dV = sdesc_sw128(base + C::kRingOff, C::kBox, 1024);
      auto scores = [&](int t, int q, int slot) {  // S_t from Q tile or buffer q and the K tile in a slot
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * C::kBox + (kk & 3) * 32;
          mma_ss_elect(tmem + t * 128, dQ + ((q * C::kTileBytes + off) >> 4),
                       dK + ((slot * C::kTileBytes + off) >> 4), C::kIdescS, kk > 0 ? 1u : 0u);
        }
        mma_commit_elect(bar(kTBarS + t));
      };
      auto product = [&](int t, int slot, bool acc) {  // O_t += P_t V
#pragma unroll
        for (int kk = 0; kk < C::kTile / 16; ++kk)
          mma_ts_elect(tmem + C::kTmO + t * D, tmem + t * 128 + kk * 8, dV + ((slot * C::kTileBytes + kk * 2048) >> 4),
                       C::kIdescO, (acc || kk > 0) ? 1u : 0u);
      };
      int item = 0, seg = 0, u0 = 0, u1 = 0;  // ring items, segments with tiles, uses of P_0 and P_1
      bool ok = true;
      auto slot = [&]() -> int { return item % C::kRing; };
      auto wait_item = [&]() -> bool {
        return uniform(mbar_wait(full(item % C::kRing), (item / C::kRing) & 1, abort_flag));
      };
      auto free_item = [&]() {
        mma_commit_elect(empty(slot()));
        ++item;
      };
      auto wait_p = [&](int t) -> bool {
        int& u = t ? u1 : u0;
        const bool got = uniform(mbar_wait(bar(kTBarP + t), u & 1, abort_flag));
        ++u;
        return got;
      };
      do {
        int jlo, jhi;
        seen_tiles<C::kRows, C::kTile, PREFIX>(p, w, jlo, jhi);
        const int n = jhi - jlo;
        if (n == 0) continue;
        if constexpr (PAIR) {
          ok = uniform(mbar_wait(bar(kTBarQ + 0), seg & 1, abort_flag)) &&
               uniform(mbar_wait(bar(kTBarQ + 1), seg & 1, abort_flag)) && wait_item();
          if (!ok) break;
          tc_fence_after();
          scores(0, 0, slot());
          scores(1, 1, slot());
          if (n == 1) mma_commit_elect(bar(kTBarQFree));
          free_item();
          for (int i = 0; i < n; ++i) {
            // the V tile, then the next K tile (if any): their items lie side by side
            const int sv = slot(), sk = (item + 1) % C::kRing;
            const bool more = i + 1 < n;
            ok = wait_item();
            if (ok && more)
              ok = uniform(mbar_wait(full(sk), ((item + 1) / C::kRing) & 1, abort_flag));
            ok = ok && wait_p(0);
            if (!ok) break;
            tc_fence_after();
            product(0, sv, i > 0);
            if (more) scores(0, 0, sk);
            else mma_commit_elect(bar(kTBarFinal + 0));
            ok = wait_p(1);
            if (!ok) break;
            tc_fence_after();
            product(1, sv, i > 0);
            mma_commit_elect(empty(sv));
            ++item;
            if (more) {
              scores(1, 1, sk);
              if (i + 2 == n) mma_commit_elect(bar(kTBarQFree));
              free_item();
            } else {
              mma_commit_elect(bar(kTBarFinal + 1));
            }
          }
        } else {
          const int q = seg & 1;
          ok = uniform(mbar_wait(bar(kTBarQ + q), (seg >> 1) & 1, abort_flag));
          for (int i = 0; ok && i < min(n, 2); ++i) {
            ok = wait_item();
            if (!ok) break;
            tc_fence_after();
            scores(i, q, slot());
            if (i + 1 == n) mma_commit_elect(bar(kTBarQFree + q));
            free_item();
          }
          // O is overwritten: the segment before has to have read it
          ok = ok && (seg == 0 || uniform(mbar_wait(bar(kTBarEpi), (seg - 1) & 1, abort_flag)));
          for (int i = 0; ok && i < n; ++i) {
            ok = wait_item() && wait_p(i & 1);
            if (!ok) break;
            tc_fence_after();
            product(i & 1, slot(), i > 1);
            if (i + 1 == n) mma_commit_elect(bar(kTBarFinal));
            free_item();
            if (i + 2 < n) {
              ok = wait_item();
              if (!ok) break;
              tc_fence_after();
              scores(i & 1, q, slot());
              if (i + 3 == n) mma_commit_elect(bar(kTBarQFree + q));
              free_item();
            }
          }
        }
        ++seg;
      } while (ok && S::next(p, w));
      if (!ok) failed(4u);
      mma_commit_elect(bar(kTBarDrain));  // flips once every MMA issued so far has completed
      mbar_wait(bar(kTBarDrain), 0, nullptr);
    } else {
      // ======================= Q loader ======================================
      const int tid = static_cast<int>(threadIdx.x) - 320;
      int seg = 0;
      bool ok = true;
      do {
        int jlo, jhi;
        seen_tiles<C::kRows, C::kTile, PREFIX>(p, w, jlo, jhi);
        if (jhi == jlo) continue;
        const int q = PAIR ? 0 : seg & 1;           // first buffer it fills
        const int use = PAIR ? seg : seg >> 1;      // earlier segments that used it
        ok = uniform(mbar_wait(bar(kTBarQFree + q), (use & 1) ^ 1, abort_flag));
        if (!ok) break;
        // asynchronous 16-byte copies, all of the block's rows in flight at once.  Each lane finds its rows
        // (32 to a warp and turn), then D / 8 lanes together copy one row, so that a copy instruction touches
        // whole 128-byte lines (one row per lane touched 32 lines each: Q took 4.6 us to arrive, not 1.9).
        constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes;
        const int half = tid >> 5;
        long long row[C::kRows / 64];
#pragma unroll
        for (int i = 0; i < C::kRows / 64; ++i) {
          int b, rr;
          row[i] = S::row(p, w, 64 * i + tid, b, rr);
        }
#pragma unroll
        for (int i = 0; i < C::kRows / 64; ++i) {
#pragma unroll 4
          for (int s = 0; s < 32; s += kAtOnce) {
            const int from = s + lane / kLanes, e = lane % kLanes, r = 64 * i + 32 * half + from;
            const long long src = __shfl_sync(0xffffffffu, row[i], from);
            if (src >= 0)  // a row that does not exist keeps what it holds: nothing of it is used
              cp_async16(base + (PAIR ? r >> 7 : q) * C::kTileBytes + (r & 127) * 128 + (e >> 3) * C::kBox +
                             (((e & 7) ^ (r & 7)) << 4),
                         p.q + src * D + e * 8);
          }
        }
        cp_async_wait_all();
        fence_proxy_async_smem();
        mbar_arrive(bar(kTBarQ + q));
        if (PAIR) mbar_arrive(bar(kTBarQ + 1));
        ++seg;
      } while (S::next(p, w));
      if (!ok) failed(32u);
    }
  } else {
    regs_inc<C::kRegSoftmax>();
    // ================= softmax, correction, epilogue ========================
    const int t = warp >> 2;  // warpgroup
    const int r = static_cast<int>(threadIdx.x) & 127;  // TMEM lane
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t tS = lane_base + t * 128;
    const uint32_t tO = lane_base + C::kTmO + t * D;
    const float c = p.scale_log2;
    const float NEG_INF = -__int_as_float(0x7f800000);
    float2* const stats = reinterpret_cast<float2*>(tile_smem + C::kStatOff);
    // The walk lies in shared memory while the tile loop runs: the S row takes 128 registers, and a walk kept
    // beside it was spilled and reloaded for every tile (2 x 256 tokens over 8192, 32/8 heads: 94 us, not 90).
    PagedWalk* const walk = reinterpret_cast<PagedWalk*>(tile_smem + C::kBarOff + kTileWalkOff) + warp;
    auto put_walk = [&](const PagedWalk& v) {
      __syncwarp();
      if (lane == 0) *walk = v;
      __syncwarp();
    };
    put_walk(w);
    int used = 0, item = 0, seg = 0;  // uses of S_t, ring items, segments with tiles
    bool ok = true, more = true;
    do {
      int n, lo, hi, k0;
      bool busy, none;            // the warp has rows that see keys; this row sees none
      bool low_edge, high_edge;  // the first or last tile reaches past the segment's keys
      {
        const PagedWalk v = *walk;
        int jlo, jhi;
        seen_tiles<C::kRows, C::kTile, PREFIX>(p, v, jlo, jhi);
        n = jhi - jlo;
        k0 = (v.tile0 + jlo) * C::kTile;
        low_edge = k0 < v.lo;
        high_edge = (v.tile0 + jhi) * C::kTile > v.hi;
        const bool there = S::row_keys(p, v, PAIR ? t * 128 + r : r, lo, hi) >= 0;
        // A row that sees no key is not masked (its warp would mask every tile) but dropped at the end, and a warp
        // of such rows has nothing to do.
        none = hi <= lo;
        if (none) lo = 0, hi = 0x7fffffff;
        busy = __any_sync(0xffffffffu, there && !none);
      }
      float m_bar = NEG_INF, l = 0.f, r_max = NEG_INF;
      if (!PAIR && t) k0 += C::kTile;
      for (int i = PAIR ? 0 : t; i < n; i += PAIR ? 1 : 2) {
        if (!uniform(mbar_wait(bar(kTBarS + t), used & 1, abort_flag))) {
          ok = false;
          break;
        }
        ++used;
        tc_fence_after();
        if (busy) {
          uint32_t s0[32], s1[32], s2[32], s3[32];
          tmem_ld32(tS + 0, s0);
          tmem_ld32(tS + 32, s1);
          tmem_ld_wait(s0);
          reg_pin(s1);
          tmem_ld32(tS + 64, s2);
          tmem_ld32(tS + 96, s3);
          float* const f0 = reinterpret_cast<float*>(s0);
          float* const f1 = reinterpret_cast<float*>(s1);
          float* const f2 = reinterpret_cast<float*>(s2);
          float* const f3 = reinterpret_cast<float*>(s3);
          const int a = lo - k0, z = hi - k0;  // columns [a, z) are visible
          const bool cut = a > 0 || z < C::kTile;
          if (cut) {
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              if (e < a || e >= z) f0[e] = NEG_INF;
              if (32 + e < a || 32 + e >= z) f1[e] = NEG_INF;
            }
          }
          float mx0 = fmax3(f0[0], f0[1], f1[0]), mx1 = fmax3(f0[2], f0[3], f1[1]);
#pragma unroll
          for (int e = 4; e < 32; e += 4) {
            mx0 = fmax3(mx0, f0[e], f0[e + 1]);
            mx1 = fmax3(mx1, f0[e + 2], f0[e + 3]);
          }
#pragma unroll
          for (int e = 2; e < 32; e += 2) {
            if (e & 2) mx0 = fmax3(mx0, f1[e], f1[e + 1]);
            else mx1 = fmax3(mx1, f1[e], f1[e + 1]);
          }
          tmem_ld_wait(s2);
          reg_pin(s3);
          if (cut) {
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              if (64 + e < a || 64 + e >= z) f2[e] = NEG_INF;
              if (96 + e < a || 96 + e >= z) f3[e] = NEG_INF;
            }
          }
          float mx2 = fmax3(f2[0], f2[1], f3[0]), mx3 = fmax3(f2[2], f2[3], f3[1]);
#pragma unroll
          for (int e = 4; e < 32; e += 4) {
            mx2 = fmax3(mx2, f2[e], f2[e + 1]);
            mx3 = fmax3(mx3, f2[e + 2], f2[e + 3]);
          }
#pragma unroll
          for (int e = 2; e < 32; e += 2) {
            if (e & 2) mx2 = fmax3(mx2, f3[e], f3[e + 1]);
            else mx3 = fmax3(mx3, f3[e], f3[e + 1]);
          }
          const float s_max = fmaxf(fmax3(mx0, mx1, mx2), mx3);
          r_max = fmaxf(r_max, s_max);
          const float m_new = s_max * c;
          const bool need = m_new > m_bar + 8.0f;  // the reference moves as in fa_fwd_kernel
          const bool any_need = __any_sync(0xffffffffu, need);
          float alpha = 1.0f;
          if (need) {
            alpha = ex2(m_bar - m_new);
            m_bar = m_new;
            l *= alpha;
          }
          const float neg_ref = m_bar == NEG_INF ? 0.f : -m_bar;
          float ls0 = 0.f, ls1 = 0.f, ls2 = 0.f, ls3 = 0.f;
          // P in bf16, the type of the product's operands (fa_paged_kernel says what that costs); l sums in fp32
          auto emit = [&](const float* f, uint32_t col) {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float x0, x1;
              fma2(x0, x1, f[2 * e], f[2 * e + 1], c, neg_ref);
              const float e0 = ex2(x0), e1 = ex2(x1);
              if (e & 1) add2(ls2, ls3, e0, e1);
              else add2(ls0, ls1, e0, e1);
              pk[e] = pack_bf16(e0, e1);
            }
            tmem_st16(tS + col, pk);
          };
          emit(f0, 0);
          emit(f1, 16);
          emit(f2, 32);
          emit(f3, 48);
          l += (ls0 + ls1) + (ls2 + ls3);
          // the warpgroup's product before this one is complete: this S was issued after it
          if (any_need && i > (PAIR ? 0 : t)) {
#pragma unroll
            for (int cc = 0; cc < D / 32; ++cc) {
              uint32_t o[32];
              tmem_ld32(tO + cc * 32, o);
              tmem_ld_wait(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st32(tO + cc * 32, o);
            }
          }
          tmem_st_wait();
        }
        if ((low_edge && i == 0) || (high_edge && i == n - 1)) {
          // key k0 + r outside the segment's range: its V row counts as zero.  iv: V's place in the
          // producer's order.  (PAIR: both warpgroups write the same zeros, each before its own product.)
          const int iv = item + (PAIR ? 2 * i + 1 : min(2, n) + i + max(0, min(n, i + 2) - 2));
          if (!uniform(mbar_wait(full(iv % C::kRing), (iv / C::kRing) & 1, abort_flag))) {
            ok = false;
            break;
          }
          if (k0 + r < walk->lo || k0 + r >= walk->hi) {
#pragma unroll
            for (int e = 0; e < D / 8; ++e)
              st_shared_v4(slot_addr(iv % C::kRing) + (e >> 3) * C::kBox + r * 128 + (e & 7) * 16, 0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        }
        tc_fence_before();
        mbar_arrive(bar(kTBarP + t));
        k0 += PAIR ? C::kTile : 2 * C::kTile;
      }
      if (!ok) break;
      item += 2 * n;
      if (none) l = 0.f;
      // O's normaliser counts the row's largest P as rounded for P V, as in fa_fwd_kernel
      float l_o = l;
      if (l != 0.f) {  // NaN (from NaN or infinite scores) goes through, here and below
        const float e_max = ex2(fmaf(r_max, c, -m_bar));
        l_o += __uint_as_float(pack_bf16(e_max, 0.f) << 16) - e_max;
      }
      float inv = l != 0.f ? 1.0f / l_o : 0.f;
      float lb = l != 0.f ? m_bar + __log2f(l) : NEG_INF;
      float inv_other = 0.f;  // factor of the other warpgroup's O
      // which O holds keys of this row: the other is nothing but stale bits.  A factor that is zero because its keys
      // weigh nothing beside the other's still multiplies (0 * NaN is NaN).
      bool some = lb != NEG_INF, some_other = false;
      if (n > 0) {
        ok = uniform(mbar_wait(bar(kTBarFinal + (PAIR ? t : 0)), seg & 1, abort_flag));
        if (!ok) break;
        tc_fence_after();
        if constexpr (!PAIR) {
          // join the two warpgroups' key tiles.  The segment's last product is complete, so the other
          // warpgroup has read what the segment before left in `stats` (its products waited for that).
          stats[t * 128 + r] = make_float2(lb, inv);
          mbar_arrive(bar(kTBarStat));
          ok = uniform(mbar_wait(bar(kTBarStat), seg & 1, abort_flag));
          if (!ok) break;
          const float2 st = stats[(t ^ 1) * 128 + r];
          const float top = fmaxf(lb, st.x);
          const float wm = lb == NEG_INF ? 0.f : ex2(lb - top), wo = st.x == NEG_INF ? 0.f : ex2(st.x - top);
          const float sum = wm + wo;  // 0: neither has keys of this row
          some_other = st.x != NEG_INF;
          inv = wm * inv / sum;
          inv_other = wo * st.y / sum;
          lb = sum != 0.f ? top + __log2f(sum) : NEG_INF;
        }
        ++seg;
      }
      PagedWalk v = *walk;
      {
        int b, rr;
        const long long out_row = S::row(p, v, PAIR ? t * 128 + r : r, b, rr);
        long long row = out_row;
        const int to = S::target(p, v, block, first, PAIR ? t * 128 + r : r, row);
        // PAIR: the whole row; else warpgroup t's half of the columns
        constexpr int kCols = PAIR ? D : D / 2;
        const int col0 = PAIR ? 0 : t * kCols;
        uint16_t* const dst16 = p.out + row * D + col0;
        float* const dst32 = (to == 1 ? p.whole_o[PREFIX] : p.piece_o[PREFIX]) + row * D + col0;
#pragma unroll
        for (int cc = 0; cc < kCols / 32; ++cc) {
          float f[32];
          if (n > 0) {
            uint32_t o[32];
            tmem_ld32(tO + col0 + cc * 32, o);
            tmem_ld_wait(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) f[e] = some ? __uint_as_float(o[e]) * inv : 0.f;
            if constexpr (!PAIR) {
              tmem_ld32(lane_base + C::kTmO + (t ^ 1) * D + col0 + cc * 32, o);
              tmem_ld_wait(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) f[e] += some_other ? __uint_as_float(o[e]) * inv_other : 0.f;
            }
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) f[e] = 0.f;
          }
          if (out_row >= 0) {
            if (to == 0) {
#pragma unroll
              for (int h = 0; h < 4; ++h)
                *reinterpret_cast<uint4*>(dst16 + cc * 32 + h * 8) =
                    make_uint4(pack_bf16(f[8 * h], f[8 * h + 1]), pack_bf16(f[8 * h + 2], f[8 * h + 3]),
                               pack_bf16(f[8 * h + 4], f[8 * h + 5]), pack_bf16(f[8 * h + 6], f[8 * h + 7]));
            } else {
#pragma unroll
              for (int h = 0; h < 4; ++h) {  // whole 32-byte sectors: the workspace's parts are 256-byte aligned
                uint32_t v8[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v8[e] = __float_as_uint(f[8 * h + e]);
                st_global_v8(dst32 + cc * 32 + h * 8, v8);
              }
            }
          }
        }
        if (out_row >= 0 && col0 == 0) {
          if (to == 0) p.lse[row] = lb * 0.69314718055994530942f;
          else (to == 1 ? p.whole_l[PREFIX] : p.piece_l[PREFIX])[row] = lb;
        }
      }
      if (!PAIR && n > 0) {
        tc_fence_before();
        mbar_arrive(bar(kTBarEpi));
      }
      first = false;
      more = S::next(p, v);
      put_walk(v);
    } while (more);
    if (!ok) failed(1u);
  }

  // ---- teardown -------------------------------------------------------------
  tc_fence_before();
  __syncthreads();
  if (warp == C::kWarpMma) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
  paged_end(beside);
}

}  // namespace fa
