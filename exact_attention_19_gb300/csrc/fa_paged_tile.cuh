// fa_paged_tile.cuh -- paged attention for row blocks of 128 on the tcgen05
// path: the shared prefix (its row blocks run over the batch) and sequences
// with more query rows per K/V head than one warp-level block holds.
//
// One CTA owns 128 query rows and streams its share of 64-key tiles past them:
// S = Q K^T and O += P V as tcgen05 MMAs (S, P and O in TMEM, as in
// fa_fwd_kernel), K and V boxes by TMA straight from the pages.  Two CTAs share
// an SM, each with one softmax warpgroup, half the TMEM and half the shared
// memory; S is double-buffered (64 columns each), so the next tile's scores
// are computed while this tile's softmax runs, and the two CTAs fill each
// other's waits between segments.
//   warps 0-3  load Q, softmax, correction, epilogue (thread = row = TMEM lane)
//   warp 4     TMA producer: K_0 K_1 V_0 K_2 V_1 ... through one ring of slots;
//              each lane issues one page's box
//   warp 5     MMA issuer
// TMEM (256 columns): S0 [0, 64), S1 [64, 128), O [128, 128 + D); P (bf16)
// overwrites the first 32 columns of its S.
// Keys outside the segment's range (the end of a page, pages given back below a
// window) are masked in S; their V rows, which may hold anything, are zeroed in
// shared memory by the softmax warps before they hand over P (0 * NaN is NaN).
#pragma once

#include "fa_paged_kernel.cuh"

namespace fa {

template <int D>
struct TileCfg {
  static constexpr int kRows = kPrefixRows, kTile = kPagedTile;
  static constexpr int kThreads = 192, kWarpProd = 4, kWarpMma = 5;
  static constexpr int kBoxes = D / 64;
  static constexpr uint32_t kQBox = kRows * 128u, kBox = kTile * 128u;
  static constexpr uint32_t kItemBytes = kBoxes * kBox;  // one tile of K or of V
  static constexpr int kRing = D == 128 ? 5 : 10;        // 80 KB
  static constexpr uint32_t kRingOff = kBoxes * kQBox;
  static constexpr uint32_t kBarOff = kRingOff + kRing * kItemBytes;
  static constexpr uint32_t kSmemBytes = kBarOff + 512;
  static constexpr uint32_t kTmemCols = 256, kTmO = 128;
  static constexpr uint32_t kIdescS = idesc_bf16(kRows, kTile, false);
  static constexpr uint32_t kIdescO = idesc_bf16(kRows, D, true);
  static_assert(2 * (kSmemBytes + 1024) <= 233472, "two CTAs per SM");
};

// barrier slots (8 bytes each); the rest of the 512-byte block: scratch of
// paged_share at 256, TMEM base at 448, abort flag at 452
enum : int { kTBarQ = 0, kTBarS = 1, kTBarP = 3, kTBarO = 5, kTBarFinal = 6, kTBarDrain = 7, kTBarRing = 8 };
constexpr uint32_t kTileScratchOff = 256, kTileTmemOff = 448, kTileAbortOff = 452;

// The tiles [jlo, jhi) of the CTA's part that some row of the block sees.
template <int RB, bool PREFIX>
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
    jlo = max(jlo, lo / kPagedTile - w.tile0);
    jhi = max(jlo, min(jhi, (hi + kPagedTile - 1) / kPagedTile - w.tile0));
  }
}

template <int D, bool PREFIX>
__global__ void __launch_bounds__(TileCfg<D>::kThreads, 2)
    fa_paged_tile_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                         const PagedParams p) {
  using C = TileCfg<D>;
  using S = PagedSchedule<C::kRows, PREFIX>;
  extern __shared__ __align__(1024) uint8_t tile_smem[];
  const uint32_t base = smem_addr(tile_smem);  // 1024-byte aligned: the kernel has no static shared memory
  const uint32_t bar0 = base + C::kBarOff;
  auto bar = [&](int i) -> uint32_t { return bar0 + 8u * static_cast<uint32_t>(i); };
  auto full = [&](int slot) -> uint32_t { return bar(kTBarRing + slot); };
  auto empty = [&](int slot) -> uint32_t { return bar(kTBarRing + C::kRing + slot); };
  auto slot_addr = [&](int slot) -> uint32_t { return base + C::kRingOff + slot * C::kItemBytes; };
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(tile_smem + C::kBarOff + kTileTmemOff);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(tile_smem + C::kBarOff + kTileAbortOff);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto failed = [&](unsigned role) {
    *abort_flag = 1;
    atomicOr(p.status, kPagedTimeout | (role << 8));
  };

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (base & 1023u) {  // the swizzled layouts need it; the launch places it so
    if (threadIdx.x == 0) atomicOr(p.status, kPagedTimeout | (16u << 8));
    return;
  }
  PagedWalk w;
  if (!paged_share<C::kRows, PREFIX, C::kThreads>(p, reinterpret_cast<long long*>(tile_smem + C::kBarOff + kTileScratchOff),
                                                  w))
    return;
  if (threadIdx.x == 0) {
    mbar_init(bar(kTBarQ), 128);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kTBarS + i), 1);
      mbar_init(bar(kTBarP + i), 128);
    }
    mbar_init(bar(kTBarO), 1);      // after every product: one may lag behind, so it names the tile before
    mbar_init(bar(kTBarFinal), 1);  // after a segment's last product
    mbar_init(bar(kTBarDrain), 1);
    for (int i = 0; i < 2 * C::kRing; ++i) mbar_init(bar(kTBarRing + i), 1);
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == C::kWarpMma) {
    tmem_alloc(smem_addr(tmem_slot), C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto uniform = [](bool v) -> bool { return __all_sync(0xffffffffu, v); };

  if (warp == C::kWarpProd) {
    // ======================= TMA producer ===================================
    tma_prefetch_map(&tmK);
    tma_prefetch_map(&tmV);
    const int chunk_rows = min(1 << p.page_shift, C::kTile);  // keys of one box: pages below 64 take several
    const int piece = lane / C::kBoxes, x = lane % C::kBoxes;
    const bool mine = lane < C::kTile / chunk_rows * C::kBoxes;
    int item = 0;
    bool ok = true;
    do {
      int jlo, jhi;
      seen_tiles<C::kRows, PREFIX>(p, w, jlo, jhi);
      const int* const pages = S::pages(p, w);
      auto key_of = [&](int j) -> int { return (w.tile0 + j) * C::kTile + piece * chunk_rows; };
      auto wanted = [&](int k) -> bool { return mine && k < w.hi && k + chunk_rows > w.lo; };
      auto page_of = [&](int j) -> int {
        const int k = key_of(j);
        return (j < jhi && wanted(k)) ? __ldg(pages + (k >> p.page_shift)) : -1;
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
      // page indices are read two and more tiles ahead of their use
      int a = page_of(jlo), b = page_of(jlo + 1), c = page_of(jlo + 2);
      if (jlo < jhi) ok = put(&tmK, jlo, a) && (jlo + 1 >= jhi || put(&tmK, jlo + 1, b));
      for (int j = jlo; ok && j < jhi; ++j) {
        const int d = page_of(j + 3);
        ok = put(&tmV, j, a) && (j + 2 >= jhi || put(&tmK, j + 2, c));
        a = b;
        b = c;
        c = d;
      }
    } while (ok && S::next(p, w));
    if (!ok) failed(2u);
    if (*abort_flag) {  // let every copy issued land before the CTA's shared memory goes
      for (int i = max(0, item - C::kRing); i < item; ++i) uniform(mbar_wait(full(i % C::kRing), (i / C::kRing) & 1, nullptr));
    }
  } else if (warp == C::kWarpMma) {
    // ======================= MMA issuer =====================================
    const uint64_t dQ = sdesc_sw128(base, 16, 1024);
    const uint64_t dK = sdesc_sw128(base + C::kRingOff, 16, 1024);
    const uint64_t dV = sdesc_sw128(base + C::kRingOff, C::kBox, 1024);
    auto scores = [&](int buf, int slot) {
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        mma_ss_elect(tmem + buf * C::kTile, dQ + (((kk >> 2) * C::kQBox + (kk & 3) * 32) >> 4),
                     dK + ((slot * C::kItemBytes + (kk >> 2) * C::kBox + (kk & 3) * 32) >> 4), C::kIdescS,
                     kk > 0 ? 1u : 0u);
    };
    auto product = [&](int buf, int slot, bool acc) {
#pragma unroll
      for (int kk = 0; kk < C::kTile / 16; ++kk)
        mma_ts_elect(tmem + C::kTmO, tmem + buf * C::kTile + kk * 8, dV + ((slot * C::kItemBytes + kk * 2048) >> 4),
                     C::kIdescO, (acc || kk > 0) ? 1u : 0u);
    };
    int item = 0, t = 0, seg = 0;  // ring items, tiles and segments so far
    bool ok = true;
    auto wait_item = [&]() -> bool { return uniform(mbar_wait(full(item % C::kRing), (item / C::kRing) & 1, abort_flag)); };
    auto next_scores = [&](int tt) -> bool {
      if (!wait_item()) return false;
      tc_fence_after();
      scores(tt & 1, item % C::kRing);
      mma_commit_elect(bar(kTBarS + (tt & 1)));
      mma_commit_elect(empty(item % C::kRing));
      ++item;
      return true;
    };
    do {
      int jlo, jhi;
      seen_tiles<C::kRows, PREFIX>(p, w, jlo, jhi);
      const int n = jhi - jlo;
      if (n == 0) continue;
      ok = uniform(mbar_wait(bar(kTBarQ), seg & 1, abort_flag));
      ++seg;
      ok = ok && next_scores(t) && (n < 2 || next_scores(t + 1));
      for (int i = 0; ok && i < n; ++i, ++t) {
        ok = wait_item() && uniform(mbar_wait(bar(kTBarP + (t & 1)), (t >> 1) & 1, abort_flag));
        if (!ok) break;
        tc_fence_after();
        product(t & 1, item % C::kRing, i > 0);
        mma_commit_elect(bar(kTBarO));
        if (i == n - 1) mma_commit_elect(bar(kTBarFinal));
        mma_commit_elect(empty(item % C::kRing));
        ++item;
        if (i + 2 < n) ok = next_scores(t + 2);
      }
    } while (ok && S::next(p, w));
    if (!ok) failed(4u);
    mma_commit_elect(bar(kTBarDrain));  // flips once every MMA issued so far has completed
    mbar_wait(bar(kTBarDrain), 0, nullptr);
  } else {
    // ================= Q, softmax, correction, epilogue =====================
    const int r = static_cast<int>(threadIdx.x);  // row of the block = TMEM lane
    const long long first_g = w.g;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    const uint32_t tO = lane_base + C::kTmO;
    const float c = p.scale_log2;
    const float NEG_INF = -__int_as_float(0x7f800000);
    int t = 0, item = 0, seg = 0;  // tiles, ring items and segments with tiles so far
    bool ok = true;
    do {
      int jlo, jhi, lo, hi;
      seen_tiles<C::kRows, PREFIX>(p, w, jlo, jhi);
      const int n = jhi - jlo;
      const long long out_row = S::row(p, w, r, lo, hi);
      const bool busy = __any_sync(0xffffffffu, out_row >= 0);  // the warp has a row to work for
      float m_bar = NEG_INF, l = 0.f, r_max = NEG_INF;
      if (n > 0) {
        // Q row to its swizzled place: every S of the segment before has been
        // waited for, so no MMA reads the buffer any more
        if (out_row >= 0) {
          const uint4* const src = reinterpret_cast<const uint4*>(p.q + out_row * D);
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            const uint4 v = __ldg(src + i);
            st_shared_v4(base + (i >> 3) * C::kQBox + r * 128 + (((i & 7) ^ (r & 7)) << 4), v.x, v.y, v.z, v.w);
          }
        }
        fence_proxy_async_smem();
        mbar_arrive(bar(kTBarQ));
      }
      for (int i = 0; i < n; ++i, ++t) {
        const uint32_t tS = lane_base + (t & 1) * C::kTile;
        if (!uniform(mbar_wait(bar(kTBarS + (t & 1)), (t >> 1) & 1, abort_flag))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const int k0 = (w.tile0 + jlo + i) * C::kTile;
        if (busy) {
          uint32_t s0[32], s1[32];
          tmem_ld32(tS, s0);
          tmem_ld32(tS + 32, s1);
          tmem_ld_wait(s0);
          reg_pin(s1);
          float* const f0 = reinterpret_cast<float*>(s0);
          float* const f1 = reinterpret_cast<float*>(s1);
          const int a = lo - k0, z = hi - k0;  // columns [a, z) are visible
          if (a > 0 || z < C::kTile) {
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
          const float s_max = fmaxf(mx0, mx1);
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
          l += (ls0 + ls1) + (ls2 + ls3);
          if (any_need && i > 0) {
            // O may be touched once the product of the tile before is complete
            if (!uniform(mbar_wait(bar(kTBarO), (t - 1) & 1, abort_flag))) {
              ok = false;
              break;
            }
            tc_fence_after();
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
        if (warp < 2 && (k0 < w.lo || k0 + C::kTile > w.hi)) {
          // key k0 + r outside the segment's range: its V row counts as zero
          const int iv = item + min(2, n) + i + max(0, min(n, i + 2) - 2);  // V's place in the producer's order
          if (!uniform(mbar_wait(full(iv % C::kRing), (iv / C::kRing) & 1, abort_flag))) {
            ok = false;
            break;
          }
          if (k0 + r < w.lo || k0 + r >= w.hi) {
#pragma unroll
            for (int e = 0; e < D / 8; ++e)
              st_shared_v4(slot_addr(iv % C::kRing) + (e >> 3) * C::kBox + r * 128 + (e & 7) * 16, 0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        }
        tc_fence_before();
        mbar_arrive(bar(kTBarP + (t & 1)));
      }
      if (!ok) break;
      item += 2 * n;
      if (n > 0) {
        ok = uniform(mbar_wait(bar(kTBarFinal), seg & 1, abort_flag));
        ++seg;
        if (!ok) break;
        tc_fence_after();
      }
      if (busy) {
        // O's normaliser counts the row's largest P as rounded for P V, as in fa_fwd_kernel
        float l_o = l;
        if (l > 0.f) {
          const float e_max = ex2(fmaf(r_max, c, -m_bar));
          l_o += __uint_as_float(pack_bf16(e_max, 0.f) << 16) - e_max;
        }
        const float inv = l > 0.f ? 1.0f / l_o : 0.f;
        const float lb = l > 0.f ? m_bar + __log2f(l) : NEG_INF;
        long long row = out_row;
        const int to = S::target(p, w, first_g, r, row);
        uint16_t* const dst16 = p.out + row * D;
        float* const dst32 = (to == 1 ? p.whole_o[PREFIX] : p.piece_o[PREFIX]) + row * D;
#pragma unroll
        for (int cc = 0; cc < D / 32; ++cc) {
          uint32_t o[32];
          if (n > 0) {
            tmem_ld32(tO + cc * 32, o);
            tmem_ld_wait(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(l > 0.f ? __uint_as_float(o[e]) * inv : 0.f);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0u;
          }
          if (out_row >= 0) {
            if (to == 0) {
#pragma unroll
              for (int h = 0; h < 4; ++h) {
                const float* const f = reinterpret_cast<const float*>(o) + 8 * h;
                *reinterpret_cast<uint4*>(dst16 + cc * 32 + h * 8) =
                    make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
              }
            } else {
#pragma unroll
              for (int h = 0; h < 8; ++h)
                *reinterpret_cast<uint4*>(dst32 + cc * 32 + h * 4) =
                    make_uint4(o[4 * h], o[4 * h + 1], o[4 * h + 2], o[4 * h + 3]);
            }
          }
        }
        if (out_row >= 0) {
          if (to == 0) p.lse[row] = lb * 0.69314718055994530942f;
          else (to == 1 ? p.whole_l[PREFIX] : p.piece_l[PREFIX])[row] = lb;
        }
      }
    } while (S::next(p, w));
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
}

}  // namespace fa
