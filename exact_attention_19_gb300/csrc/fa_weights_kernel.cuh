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

}  // namespace fa
