// fa_paged_kernel.cuh -- attention of a few new tokens per sequence over a
// paged K/V cache, with an optional prefix that every sequence shares.
//
// Rows.  Query head h = hk * G + g reads K/V head hk (G = H / Hk); the G * T
// query rows of one (sequence, K/V head) are contiguous in [B, H, T, d] and
// share every K/V byte.  Row r of them is token t = r % T.  With len the
// sequence's own cached tokens and fresh its new ones, token t sits at own
// position len - fresh + t and sees the own keys its window reaches, and every
// prefix key at or before it.
//
// Schedule.  A work unit is one block of rows against one tile of keys; a
// launch covers either the sequences' own keys (row blocks of one sequence and
// K/V head) or the shared prefix (row blocks over all the batch's rows of a K/V
// head, so its K/V is read once for the batch and not once per sequence).  The
// units of a launch form one line and CTA c takes [c W / P, (c + 1) W / P),
// computed on the device from the lengths there, so the host needs none of them
// and a captured launch stays right as the sequences grow.  A row block is
// charged with every tile that some row of its sequence and K/V head may see; a
// CTA skips those that none of the block's own rows sees.  So shares are equal in
// work where all rows see about the same keys (decoding, a short chunk over a
// long context), and uneven where they do not (a whole prompt: its early blocks;
// padding rows): 512 / 2048 / 8192 tokens at once, 32/8 heads of 128, take 23 / 77 /
// 666 us against 2 / 18 / 291 at the tensor rate.  A CTA that holds all units of a row block writes its
// output; else it writes its part (O normalised by its own sum, and L, the
// base-2 log of that sum) and a merge kernel joins the parts:
//   L = log2 sum 2^L_i,  O = sum 2^(L_i - L) O_i.
#pragma once

#include <cstdint>
#include <type_traits>

#include <cuda.h>

#include "fa_ptx.cuh"

namespace fa {

// status word bits of the paged kernels (fa.h)
constexpr unsigned kPagedTimeout = 1u, kPagedPage = 2u;

struct PagedParams {
  const uint16_t* q;        // [B, H, T, D]
  uint16_t* out;            // [B, H, T, D]
  float* lse;               // [B, H, T]
  const int* table;         // [B, max_pages]
  const int* lens;          // [B]
  const int* new_lens;      // [B] or nullptr
  const int* prefix_pages;  // [ceil(prefix_len / page)]
  int B, Hk, T, rows;       // rows = G * T of one (sequence, K/V head)
  int n_pages, max_pages, page_shift;
  int capacity;             // tokens a row of the table can hold (clipped to an int)
  int prefix_len;           // 0: no prefix
  int left, right;          // own window, -1 = open
  float scale_log2;         // scale * log2(e)
  long long* plan;          // own units, for the merge of a large batch: [0] units, [1 + b] first unit of sequence b
  int own_grid;             // CTAs of the launch over own keys
  int rb[2];                // rows of a row block: own keys, prefix
  int prefix_blocks;        // row blocks of a K/V head, key tiles, units and CTAs of the prefix
  int prefix_tiles;
  long long prefix_units, prefix_ctas;
  // [0] own keys, [1] prefix: parts of row blocks that CTAs share, two per CTA ([2 * CTAs, row block, D]), and
  // with a prefix the row blocks that one CTA finished ([B * H * T, D])
  float* piece_o[2];
  float* piece_l[2];
  float* whole_o[2];
  float* whole_l[2];
  unsigned int* status;
};

// An index or length that an earlier kernel of the stream may have written: a coherent load that stays behind the
// wait for that kernel (paged_begin).  ld.global.nc wants memory that nothing writes while the kernel is resident,
// and as plain loads the compiler left 16 x 4 tokens over 31999 keys 2 us slower than either.
__device__ __forceinline__ int coherent(const int* at) {
  int v;
  asm volatile("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(at) : "memory");
  return v;
}

// The own keys [lo, hi) of a sequence that any of its new tokens sees.
struct SeqKeys {
  int len, fresh, lo, hi;
};
__device__ __forceinline__ SeqKeys seq_keys(const PagedParams& p, int len, int fresh) {
  SeqKeys s;
  s.len = max(0, min(len, p.capacity));
  s.fresh = max(0, min(fresh, p.T));
  s.hi = s.fresh > 0 ? s.len : 0;
  s.lo = p.left < 0 ? 0 : static_cast<int>(max(0ll, static_cast<long long>(s.len) - s.fresh - p.left));
  s.lo = min(s.lo, s.hi);
  return s;
}
__device__ __forceinline__ SeqKeys seq_keys(const PagedParams& p, int b) {
  return seq_keys(p, coherent(p.lens + b), p.new_lens ? coherent(p.new_lens + b) : p.T);
}
__device__ __forceinline__ int tiles_of(int lo, int hi, int tile) { return hi > lo ? (hi + tile - 1) / tile - lo / tile : 0; }

// Own keys [lo, hi) that one row (token t of a sequence) sees.
__device__ __forceinline__ void row_own_keys(const PagedParams& p, const SeqKeys& s, int t, int& lo, int& hi) {
  const long long pos = static_cast<long long>(s.len) - s.fresh + t;
  lo = p.left < 0 ? 0 : static_cast<int>(max(0ll, pos - p.left));
  hi = p.right < 0 ? s.len : static_cast<int>(max(0ll, min(static_cast<long long>(s.len), pos + p.right + 1)));
  if (t >= s.fresh || (p.prefix_len > 0 && pos < 0)) hi = 0;
}
// Prefix keys [0, hi) that one row sees: all of them, unless it holds no token.
__device__ __forceinline__ int row_prefix_keys(const PagedParams& p, const SeqKeys& s, int t) {
  return (t < s.fresh && s.len - s.fresh + t >= 0) ? p.prefix_len : 0;
}

// Units that a CTA takes at least: with fewer, the parts' O (rb * D * 4 bytes,
// written and read again) outweighs the keys they read (512 D bytes a tile), with
// more, short calls leave SMs idle.  Row blocks of 256: 3 for own keys (16 x 1000
// keys, 2 K/V heads: 21 us, with 8 it takes 27), 8 for a prefix, a middle: us with
// 4 / 6 / 8 / 12, 32/8 heads unless noted: 64 sequences behind 3000 tokens 28 / 30 / 34 /
// 41, behind 6000 43 / 31 / 35 / 43, behind 20000 58 / 58 / 58 / 49; 40 x 2 of 16/4 heads
// behind 12000 34 / 36 / 34 / 39; 128 x 2 of 16/16 behind 2000 65 / 52 / 43 / 43; 128 of 64/8
// (d = 64) behind 1500 33 / 33 / 28 / 36; 100 of 8/2 (d = 64) behind 8000 23 / 25 / 28 / 33.
__host__ __device__ constexpr int least_units(int rb, bool prefix) {
  return rb == 16 ? 1 : rb == 128 ? 4 : prefix ? 8 : 3;
}
__host__ __device__ __forceinline__ long long paged_ctas(long long grid, long long units, int least) {
  const long long most = units / least;
  return most < 1 ? 1 : (most < grid ? most : grid);
}
// a / b for a >= 0, b > 0: a 32-bit division where both fit (a 64-bit one is a long instruction sequence)
__device__ __forceinline__ long long quotient(long long a, long long b) {
  if ((static_cast<unsigned long long>(a | b) >> 32) == 0) return static_cast<unsigned>(a) / static_cast<unsigned>(b);
  return a / b;
}
__device__ __forceinline__ long long cta_start(long long units, long long ctas, long long c) {
  return quotient(c * units, ctas);
}
__device__ __forceinline__ long long cta_of(long long units, long long ctas, long long x) {
  return quotient((x + 1) * ctas - 1, units);
}
__host__ __device__ __forceinline__ int row_blocks(long long rows, int rb) { return static_cast<int>((rows + rb - 1) / rb); }

// Programmatic dependent launch.  Every kernel here is launched so that it may
// be scheduled before the one ahead of it on the stream has finished, and
// paged_begin waits for that (inputs and workspace are then as stream order
// has them) before it lets the next one be scheduled.  The own-key kernel behind
// a prefix kernel needs nothing of it and runs beside it (all work before the
// prefix kernel is done, or that kernel would not have let this one start); it
// waits before it ends, so that the merge, which waits for it, sees both.
// `beside`: this is such a kernel.
// Everything that an earlier kernel of the stream may write (queries, lengths, page indices, parts) is read by
// coherent loads behind the wait.  (The merge's lengths: RowParts::wait.)
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void paged_begin(bool beside) {
  if (!beside) grid_wait();
  grid_release();
}
__device__ __forceinline__ void paged_end(bool beside) {
  if (beside) grid_wait();
}

constexpr int kPagedTile = 128;  // keys of a unit

// What a row block costs beside its tiles (its rows, its first wait, its
// output), in tiles: the line of units holds so many empty ones behind each row
// block's, so that shares of many short row blocks are not the last to finish.
__host__ __device__ constexpr int extra_units(int rb) { return rb == 16 ? 1 : 4; }

// A row block against the tiles of its keys that this CTA holds.
struct PagedWalk {
  long long g, gend;  // first unit of the current segment part, end of the CTA's units
  int b, hk, rb;      // sequence (own keys), K/V head, row block
  int tile0, n;       // first key tile of the row block and their number
  int j, jend;        // the part of them this CTA holds
  int lo, hi;         // keys that any row of the segment may see
};

template <int RB, int TILE, bool PREFIX>
struct PagedSchedule {
  static constexpr int kExtra = extra_units(RB);
  // units of a row block of n tiles
  static __device__ __forceinline__ int units(int n) { return n > 0 ? n + kExtra : 0; }
  static __device__ __forceinline__ int blocks(const PagedParams& p) {
    return PREFIX ? p.prefix_blocks : row_blocks(p.rows, RB);
  }
  static __device__ __forceinline__ void enter_seq(const PagedParams& p, PagedWalk& w) {
    for (;; ++w.b) {  // w.g < w.gend, so a sequence with units follows
      const SeqKeys s = seq_keys(p, w.b);
      w.lo = s.lo;
      w.hi = s.hi;
      w.tile0 = s.lo / TILE;
      w.n = tiles_of(s.lo, s.hi, TILE);
      if (w.n > 0 || w.b + 1 >= p.B) return;
    }
  }
  static __device__ __forceinline__ void part(PagedWalk& w) {
    w.jend = static_cast<int>(min(static_cast<long long>(w.n), w.j + (w.gend - w.g)));
  }
  static __device__ __forceinline__ void next_block(const PagedParams& p, PagedWalk& w) {
    w.j = 0;
    if (++w.rb == blocks(p)) {
      w.rb = 0;
      if (++w.hk == p.Hk) {
        w.hk = 0;
        ++w.b;
        if (!PREFIX) enter_seq(p, w);
      }
    }
  }
  // first segment of the units [g, gend), g < gend; b, b_unit: the sequence that holds g and its first
  // unit (own keys).  starts: it holds unit g.  False: the units are empty ones.
  static __device__ __forceinline__ bool begin(const PagedParams& p, PagedWalk& w, long long g, long long gend, int b,
                                               long long b_unit, bool& starts) {
    w.g = g;
    w.gend = gend;
    w.b = b;
    if constexpr (PREFIX) {
      w.n = p.prefix_tiles;
      w.tile0 = 0;
      w.lo = 0;
      w.hi = p.prefix_len;
    } else {
      enter_seq(p, w);
    }
    const int each = units(w.n);
    const long long i = quotient(g - b_unit, each);
    w.j = static_cast<int>((g - b_unit) - i * each);
    w.hk = static_cast<int>(quotient(i, blocks(p)));
    w.rb = static_cast<int>(i - static_cast<long long>(w.hk) * blocks(p));
    starts = w.j < w.n;
    if (!starts) {
      w.g += each - w.j;
      if (w.g >= w.gend) return false;
      next_block(p, w);
    }
    part(w);
    return true;
  }
  // the segment after the current one, w.j still its first tile; false: none left
  static __device__ __forceinline__ bool next(const PagedParams& p, PagedWalk& w) {
    w.g += w.jend - w.j + (w.jend == w.n ? kExtra : 0);
    if (w.g >= w.gend) return false;
    next_block(p, w);
    part(w);
    return true;
  }
  // page indices of the segment's keys
  static __device__ __forceinline__ const int* pages(const PagedParams& p, const PagedWalk& w) {
    return PREFIX ? p.prefix_pages : p.table + static_cast<long long>(w.b) * p.max_pages;
  }
  // The row of [B * H * T] that row r of the segment's block is (-1: none): row rr of sequence b and the
  // segment's K/V head.
  static __device__ __forceinline__ long long row(const PagedParams& p, const PagedWalk& w, int r, int& b, int& rr) {
    b = w.b;
    rr = w.rb * RB + r;
    bool there = rr < p.rows;
    if constexpr (PREFIX) {
      b = rr / p.rows;
      rr -= b * p.rows;
      there = b < p.B;
    }
    return there ? (static_cast<long long>(b) * p.Hk + w.hk) * p.rows + rr : -1;
  }
  // The same with the keys [lo, hi) that the row sees; a row that does not exist needs no mask, as nothing of it
  // is stored.
  static __device__ __forceinline__ long long row_keys(const PagedParams& p, const PagedWalk& w, int r, int& lo,
                                                       int& hi) {
    int b, rr;
    const long long at = row(p, w, r, b, rr);
    lo = 0;
    hi = 0x7fffffff;
    if (at < 0) return at;
    if constexpr (PREFIX) hi = row_prefix_keys(p, seq_keys(p, b), rr % p.T);
    else row_own_keys(p, seq_keys(p, b), rr % p.T, lo, hi);
    return at;
  }
  // where a row block's result goes: 0 the output, 1 whole_*, 2 piece_* (row = of the piece); first: the
  // segment holds the CTA's first unit
  static __device__ __forceinline__ int target(const PagedParams& p, const PagedWalk& w, int block, bool first, int r,
                                               long long& row) {
    if (w.jend - w.j == w.n) return p.prefix_len > 0 ? 1 : 0;
    const long long slot = 2ll * block + (first ? 0 : 1);
    row = slot * RB + r;
    return 2;
  }
};

// ---------------------------------------------------------------------------
// Row blocks of 16: warp-level MMAs.
// ---------------------------------------------------------------------------
// Decoding is bound by reading K and V once: 2 D multiply-adds per row and
// 2-byte element leave a block of 16 rows far below the tensor rate, so the
// warp-level m16n8k16 MMA (fed from registers) carries it, and each warp runs
// alone: it streams its own 32 keys of every 128-key tile through its own ring
// of TMA boxes, holds its own running maximum, sum and O accumulator, and meets
// the other warps only at the end of a row block.  No barrier between warps
// stands in the loop, so their waits overlap.  With eight warps on an SM the
// instructions per key matter: 32 keys to a step, not 16, and the page indices
// of 32 steps held by the lanes (32 sequences of up to 8192 keys, 32/8 heads of
// 128, 556 MB: 93.6 us, with 16 keys 98.5).
// Bound: DRAM.  The same case now takes 90 us, 6.2 TB/s, 91% of the copy rate; SMs
// reach DRAM at unequal rates, so equal shares end between 61 and 91 us.  Shares
// that CTAs take over from one another (cluster launch control) were slower, 99
// us for 93.6, as each one's end and start costs about 2 us of a CTA; so were warps
// as workers of their own (92.5 for 90.7).  Short calls (8 x 1000 keys: 9 us) are
// bound by the chain of loads: lengths, page index, keys, then the merge.
template <int D>
struct PagedCfg {
  static constexpr int kWarps = 4, kThreads = 128;
  static constexpr int kRows = 16, kKeys = 32, kTile = kPagedTile;
  static_assert(kTile == kWarps * kKeys, "a warp takes its keys of every tile");
  static constexpr int kBoxes = D / 64;
  static constexpr uint32_t kBoxBytes = kKeys * 128u;
  static constexpr uint32_t kItemBytes = kBoxes * kBoxBytes;  // 32 keys of K or of V
  static constexpr int kRing = D == 128 ? 3 : 6;              // items per warp: 24 KB
  static constexpr uint32_t kRingBytes = kWarps * kRing * kItemBytes;
  static constexpr int kMergeStride = 40;  // floats of a row in the merge buffer: 32 columns at a time, + 8 spreads
                                           // the rows over the banks
  static constexpr uint32_t kMergeOff = kRingBytes;
  static constexpr uint32_t kStatOff = kMergeOff + kWarps * 16 * kMergeStride * 4;
  static constexpr uint32_t kBarOff = kStatOff + kWarps * 16 * 8;
  static constexpr uint32_t kSmemBytes = kBarOff + kWarps * kRing * 8 + 128 + 1024;  // + alignment slack
  static_assert(2 * (kSmemBytes + 1024) <= 233472, "two CTAs per SM");
};

// TMA tile load from a 4-D map (d, token of the page, K/V head, page).  A page
// index outside the map loads zeros.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z,
                                            int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_t(uint32_t addr, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
               : "r"(addr)
               : "memory");
}
// c[16 x 8] += a[16 x 16] b[16 x 8], bf16 in, fp32 accumulators
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Block-wide: share `block` of the prefix's or the own keys' units, as the walk's
// first segment; false when it has none.  For own keys the units come from the
// lengths, and share 0 leaves the plan for the merge.
template <int RB, int TILE, bool PREFIX, int THREADS>
__device__ __forceinline__ bool paged_share(const PagedParams& p, const int block,
                                            long long* scratch /* shared, THREADS / 32 + 2 */, PagedWalk& w,
                                            bool& starts) {
  using S = PagedSchedule<RB, TILE, PREFIX>;
  if constexpr (PREFIX) {
    if (block >= p.prefix_ctas) return false;
    const long long g = cta_start(p.prefix_units, p.prefix_ctas, block);
    return S::begin(p, w, g, cta_start(p.prefix_units, p.prefix_ctas, block + 1ll), 0, 0, starts);
  } else {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int kWarps = THREADS / 32;
    const long long per = static_cast<long long>(p.Hk) * S::blocks(p);
    long long g = 0, gend = 0;
    // pass 0 sums, pass 1 finds the sequence that holds unit g (from what pass 0 left in the registers
    // when every sequence has a thread)
    long long first = 0, mine = 0;
    for (int pass = 0; pass < 2; ++pass) {
      long long run = 0;
      for (int b0 = 0; b0 < p.B; b0 += THREADS) {
        const int b = b0 + static_cast<int>(threadIdx.x);
        if (pass == 1 && p.B <= THREADS) {
          if (mine > 0 && first <= g && g < first + mine) {
            scratch[kWarps] = b;
            scratch[kWarps + 1] = first;
          }
          __syncthreads();
          break;
        }
        mine = 0;
        if (b < p.B) {
          const SeqKeys s = seq_keys(p, b);
          mine = per * S::units(tiles_of(s.lo, s.hi, TILE));
          if (pass == 0 && block == 0 && coherent(p.lens + b) > p.capacity) atomicOr(p.status, kPagedPage);
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
        first = before + incl - mine;
        if (pass == 0 && block == 0 && b < p.B) p.plan[1 + b] = first;
        if (pass == 1 && mine > 0 && first <= g && g < first + mine) {
          scratch[kWarps] = b;
          scratch[kWarps + 1] = first;
        }
        run += all;
        __syncthreads();
      }
      if (pass == 0) {
        const long long ctas = paged_ctas(p.own_grid, run, least_units(RB, false));
        if (block == 0 && threadIdx.x == 0) {
          p.plan[0] = run;
          p.plan[1 + p.B] = run;
        }
        if (block >= ctas) return false;
        g = cta_start(run, ctas, block);
        gend = cta_start(run, ctas, block + 1ll);
        if (g >= gend) return false;
      }
    }
    return S::begin(p, w, g, gend, static_cast<int>(scratch[kWarps]), scratch[kWarps + 1], starts);
  }
}

// The CTA's share `block` of the prefix or of the own keys.
template <int D, bool PREFIX>
__device__ __forceinline__ void paged_rows(const CUtensorMap& tmK, const CUtensorMap& tmV, const PagedParams& p,
                                           const int block, uint8_t* const smem_raw, long long* const scratch,
                                           const bool beside) {
  using C = PagedCfg<D>;
  using S = PagedSchedule<C::kRows, C::kTile, PREFIX>;
  constexpr int kNT = D / 8;   // 8-column tiles of O
  constexpr int kKT = D / 16;  // 16-deep steps of Q K^T
  const uint32_t raw_addr = smem_addr(smem_raw);
  const uint32_t base = (raw_addr + 1023u) & ~1023u;
  uint8_t* const sbase = smem_raw + (base - raw_addr);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(sbase + C::kBarOff + C::kWarps * C::kRing * 8);
  const uint32_t bars = base + C::kBarOff + warp * C::kRing * 8;  // this warp's ring
  const uint32_t ring = base + warp * C::kRing * C::kItemBytes;
  float* const merge = reinterpret_cast<float*>(sbase + C::kMergeOff);
  float* const stat = reinterpret_cast<float*>(sbase + C::kStatOff);  // [warp][16 rows][m, l]

  if (lane == 0) {
    for (int i = 0; i < C::kRing; ++i) mbar_init(bars + 8 * i, 1);
    if (warp == 0) *abort_flag = 0;
    mbar_init_fence();
    tma_prefetch_map(&tmK);
    tma_prefetch_map(&tmV);
  }
  paged_begin(beside);
  PagedWalk w;
  bool first;  // the segment holds the share's first unit
  if (!paged_share<C::kRows, C::kTile, PREFIX, C::kThreads>(p, block, scratch, w, first)) {
    paged_end(beside);
    return;
  }
  __syncthreads();

  // the tiles [j0, j1) of a segment part in which this warp has keys
  auto mine = [&](const PagedWalk& v, int from, int& j0, int& j1) {
    const int k = v.tile0 * C::kTile + warp * C::kKeys;  // first key in the segment's first tile
    j0 = max(from, k + C::kKeys > v.lo ? 0 : 1);
    j1 = min(v.jend, (max(v.hi - k, 0) + C::kTile - 1) / C::kTile);
  };

  // ---- this warp's stream of TMA items -----------------------------------
  // The fetch side walks the same segments ahead of the products, up to 32
  // steps (of one K and one V item) at a time: lane i holds the page indices of
  // step i, and those of the 32 after them are being read meanwhile.
  const int chunk = min(1 << p.page_shift, C::kKeys);  // keys of a box: a step takes two of pages of 16
  const int half = lane / C::kBoxes, box = lane % C::kBoxes;
  const bool issues = lane < C::kKeys / chunk * C::kBoxes;
  PagedWalk f = w;
  int f_from = w.j;
  int f_i = 0, f_n = 0, f_key = 0, f_hk = 0, f_lo = 0, f_hi = 0, f_page = 0, f_page2 = 0;  // steps being fetched
  int n_n = 0, n_key = 0, n_hk = 0, n_lo = 0, n_hi = 0, n_page = 0, n_page2 = 0;           // the ones after them
  bool f_more = true;
  auto advance = [&]() {
    f_i = 0;
    f_n = n_n;
    f_key = n_key;
    f_hk = n_hk;
    f_lo = n_lo;
    f_hi = n_hi;
    f_page = n_page;
    f_page2 = n_page2;
    n_n = 0;
    while (f_more) {
      int j0, j1;
      mine(f, f_from, j0, j1);
      if (j0 < j1) {
        n_n = min(32, j1 - j0);
        n_key = (f.tile0 + j0) * C::kTile + warp * C::kKeys;
        n_hk = f.hk;
        n_lo = f.lo;
        n_hi = f.hi;
        f_from = j0 + n_n;
        const int k = n_key + lane * C::kTile;
        const int* const pages = S::pages(p, f);
        n_page = n_page2 = -1;
        if (lane < n_n) {
          if (k + chunk > f.lo) n_page = coherent(pages + (k >> p.page_shift));
          if (chunk < C::kKeys && k + chunk < f.hi) n_page2 = coherent(pages + (k >> p.page_shift) + 1);
        }
        return;
      }
      f_more = S::next(p, f);
      f_from = f.j;
    }
  };
  int f_slot = 0, issued = 0, consumed = 0;
  auto fetch = [&](auto what) {  // the next item into f_slot, which is free
    constexpr bool is_v = decltype(what)::value;
    if (f_i >= f_n) return;
    const uint32_t bar = bars + 8 * f_slot;
    const int page_a = __shfl_sync(0xffffffffu, f_page, f_i), page_b = __shfl_sync(0xffffffffu, f_page2, f_i);
    const int key = f_key + f_i * C::kTile + half * chunk, page = half ? page_b : page_a;
    const bool wanted = issues && key < f_hi && key + chunk > f_lo;
    const unsigned boxes = __popc(__ballot_sync(0xffffffffu, wanted));
    if (lane == 0) mbar_arrive_expect_tx(bar, boxes * chunk * 128u);
    if (wanted) {
      if (!is_v && static_cast<unsigned>(page) >= static_cast<unsigned>(p.n_pages)) atomicOr(p.status, kPagedPage);
      tma_load_4d(ring + f_slot * C::kItemBytes + box * C::kBoxBytes + half * chunk * 128, is_v ? &tmV : &tmK, bar,
                  box * 64, key & ((1 << p.page_shift) - 1), f_hk, page);
    }
    ++issued;
    f_slot = f_slot + 1 == C::kRing ? 0 : f_slot + 1;
    if constexpr (is_v) {
      if (++f_i == f_n) advance();
    }
  };
  constexpr std::false_type kItemK{};
  constexpr std::true_type kItemV{};
  advance();
  advance();
  // the ring is filled in the order K V K V ...; the products free a K item, then a V item, so with an odd
  // ring a freed K makes room for a V and the other way round
#pragma unroll 1
  for (int i = 0; i < C::kRing / 2; ++i) {
    fetch(kItemK);
    fetch(kItemV);
  }
  if constexpr (C::kRing % 2) fetch(kItemK);

  int c_slot = 0;
  uint32_t c_phase = 0;
  bool ok = true;
  auto wait_item = [&]() -> uint32_t {  // address of the next item once it has landed
    if (ok) {
      ok = __all_sync(0xffffffffu, mbar_wait(bars + 8 * c_slot, c_phase, abort_flag));
      if (!ok) {
        *abort_flag = 1;
        if (lane == 0) atomicOr(p.status, kPagedTimeout | (1u << 8));
      }
    }
    return ring + c_slot * C::kItemBytes;
  };
  auto free_item = [&](auto next_is_v) {
    if (ok) {
      ++consumed;
      __syncwarp();
      fetch(next_is_v);
    }
    if (++c_slot == C::kRing) {
      c_slot = 0;
      c_phase ^= 1u;
    }
  };

  const float NEG_INF = -__int_as_float(0x7f800000);
  const int g8 = lane >> 2, q4 = lane & 3;  // this thread's rows g8, g8 + 8 and columns 2 q4, 2 q4 + 1
  do {
    // ---- the segment's rows ------------------------------------------------
    int lo[2], hi[2];
    uint32_t qf[kKT][4];
    long long out_row[2];  // row in [B * H * T], -1: no such row
    bool none[2];          // the row sees no key
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      out_row[i] = S::row_keys(p, w, g8 + 8 * i, lo[i], hi[i]);
      const bool there = out_row[i] >= 0;
      none[i] = hi[i] <= lo[i];  // such a row is not masked either (its warp would mask every tile), but dropped
      if (none[i]) lo[i] = 0, hi[i] = 0x7fffffff;
      const uint32_t* const src = reinterpret_cast<const uint32_t*>(p.q + (there ? out_row[i] : 0) * D);
#pragma unroll
      for (int kk = 0; kk < kKT; ++kk) {
        qf[kk][i] = there ? src[kk * 8 + q4] : 0u;
        qf[kk][2 + i] = there ? src[kk * 8 + 4 + q4] : 0u;
      }
    }
    float o[kNT][4];
#pragma unroll
    for (int i = 0; i < kNT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float m[2] = {NEG_INF, NEG_INF}, l[2] = {0.f, 0.f};  // base-2 scaled units; l: this thread's share

    int j0, j1;
    mine(w, w.j, j0, j1);
    for (int j = j0; j < j1; ++j) {
      const int k0 = (w.tile0 + j) * C::kTile + warp * C::kKeys;
      // S = Q K^T over 32 keys
      const uint32_t kt = wait_item();
      float s[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
      const int mi = lane >> 3, r8 = lane & 7;
      if (ok) {
        const int row = (mi >> 1) * 8 + r8;  // key (and key + 16)
#pragma unroll
        for (int kk = 0; kk < kKT; ++kk) {
          const uint32_t chunk16 = static_cast<uint32_t>((kk & 3) * 2 + (mi & 1));
          const uint32_t at = kt + (kk >> 2) * C::kBoxBytes + row * 128 + ((chunk16 ^ static_cast<uint32_t>(row & 7)) << 4);
          uint32_t b0, b1, b2, b3;
          ldmatrix4(at, b0, b1, b2, b3);
          mma16816(s[0], qf[kk], b0, b1);
          mma16816(s[1], qf[kk], b2, b3);
          ldmatrix4(at + 16 * 128, b0, b1, b2, b3);
          mma16816(s[2], qf[kk], b0, b1);
          mma16816(s[3], qf[kk], b2, b3);
        }
      }
      free_item(std::integral_constant<bool, C::kRing % 2 != 0>{});
      // masks: rows' own bounds
      const bool cut = k0 < max(lo[0], lo[1]) || k0 + C::kKeys > min(hi[0], hi[1]);
      if (__any_sync(0xffffffffu, cut)) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = k0 + i * 8 + q4 * 2 + (e & 1);
            if (key < lo[e >> 1] || key >= hi[e >> 1]) s[i][e] = NEG_INF;
          }
      }
      float m_new[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float mx = fmaxf(fmax3(s[0][2 * i], s[0][2 * i + 1], s[1][2 * i]), fmax3(s[1][2 * i + 1], s[2][2 * i], s[2][2 * i + 1]));
        mx = fmax3(mx, s[3][2 * i], s[3][2 * i + 1]);
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        m_new[i] = fmaxf(m[i], mx * p.scale_log2);
      }
      // the running maximum is exact here (no threshold), so the largest
      // probability of a row is 1 and its bf16 rounding is exact
      if (__any_sync(0xffffffffu, m_new[0] > m[0] || m_new[1] > m[1])) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float alpha = m[i] == NEG_INF ? 0.f : ex2(m[i] - m_new[i]);
          m[i] = m_new[i];
          l[i] *= alpha;
#pragma unroll
          for (int n = 0; n < kNT; ++n) {
            o[n][2 * i] *= alpha;
            o[n][2 * i + 1] *= alpha;
          }
        }
      }
      // P in bf16, the type the product takes beside V's, as in fa_fwd: O is off by about half a bf16 step more than
      // with P in fp32 (2.0e-3 for 1.7e-3 of its size against 64 bits); l sums the unrounded values
      uint32_t pf[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float ref = m[i] == NEG_INF ? 0.f : -m[i];
        float sum = 0.f;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const float e0 = ex2(fmaf(s[n][2 * i], p.scale_log2, ref)), e1 = ex2(fmaf(s[n][2 * i + 1], p.scale_log2, ref));
          sum += e0 + e1;
          pf[n >> 1][(n & 1) * 2 + i] = pack_bf16(e0, e1);
        }
        l[i] += sum;
      }
      // O += P V; keys outside the segment's range may hold anything (the end
      // of a page, a page given back): their V counts as zero, as 0 * NaN would not
      const uint32_t vt = wait_item();
      if (ok) {
        const int row = (mi & 1) * 8 + r8;  // key (and key + 16)
        auto product = [&](auto edge) {
          constexpr bool masked = decltype(edge)::value;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t keep[2] = {0xffffffffu, 0xffffffffu};
            if constexpr (masked) {
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const int key = k0 + h * 16 + i * 8 + q4 * 2;
                keep[i] = ((key >= w.lo && key < w.hi) ? 0xffffu : 0u) |
                          ((key + 1 >= w.lo && key + 1 < w.hi) ? 0xffff0000u : 0u);
              }
            }
#pragma unroll
            for (int n = 0; n < kNT; n += 2) {
              uint32_t b0, b1, b2, b3;
              const uint32_t chunk16 = static_cast<uint32_t>((n & 7) + (mi >> 1));
              ldmatrix4_t(vt + (n >> 3) * C::kBoxBytes + (h * 16 + row) * 128 +
                              ((chunk16 ^ static_cast<uint32_t>(row & 7)) << 4),
                          b0, b1, b2, b3);
              if constexpr (masked) b0 &= keep[0], b1 &= keep[1], b2 &= keep[0], b3 &= keep[1];
              mma16816(o[n], pf[h], b0, b1);
              mma16816(o[n + 1], pf[h], b2, b3);
            }
          }
        };
        if (k0 < w.lo || k0 + C::kKeys > w.hi) product(std::true_type{});
        else product(std::false_type{});
      }
      free_item(std::integral_constant<bool, C::kRing % 2 == 0>{});
    }

    // ---- join the four warps: each ends with D / 4 columns of all rows ----
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
    }
    // This warp keeps the upper (or lower) half of its columns and gets the
    // other warp's values of them, 32 columns at a time.
    auto exchange = [&](const int other, const bool upper, auto& from, auto& to, auto half_tiles) {
      constexpr int kHalf = decltype(half_tiles)::value, kStep = kHalf < 4 ? kHalf : 4;
      float* const out = merge + warp * 16 * C::kMergeStride;
      const float* const theirs = merge + other * 16 * C::kMergeStride;
      float a[2], c[2];
#pragma unroll
      for (int n0 = 0; n0 < kHalf; n0 += kStep) {
        __syncthreads();  // the buffer is free
#pragma unroll
        for (int n = 0; n < kStep; ++n) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float x = upper ? from[n0 + n][2 * i] : from[kHalf + n0 + n][2 * i];
            const float y = upper ? from[n0 + n][2 * i + 1] : from[kHalf + n0 + n][2 * i + 1];
            *reinterpret_cast<float2*>(out + (g8 + 8 * i) * C::kMergeStride + n * 8 + 2 * q4) = make_float2(x, y);
          }
        }
        if (n0 == 0 && q4 == 0) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
            *reinterpret_cast<float2*>(stat + (warp * 16 + g8 + 8 * i) * 2) = make_float2(m[i], l[i]);
        }
        __syncthreads();
        if (n0 == 0) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float2 ml = *reinterpret_cast<const float2*>(stat + (other * 16 + g8 + 8 * i) * 2);
            const float m_new = fmaxf(m[i], ml.x);
            a[i] = m[i] == NEG_INF ? 0.f : ex2(m[i] - m_new);
            c[i] = ml.x == NEG_INF ? 0.f : ex2(ml.x - m_new);
            m[i] = m_new;
            l[i] = a[i] * l[i] + c[i] * ml.y;
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int n = 0; n < kStep; ++n) {
            const float2 t = *reinterpret_cast<const float2*>(theirs + (g8 + 8 * i) * C::kMergeStride + n * 8 + 2 * q4);
            const float x = upper ? from[kHalf + n0 + n][2 * i] : from[n0 + n][2 * i];
            const float y = upper ? from[kHalf + n0 + n][2 * i + 1] : from[n0 + n][2 * i + 1];
            to[n0 + n][2 * i] = a[i] * x + c[i] * t.x;
            to[n0 + n][2 * i + 1] = a[i] * y + c[i] * t.y;
          }
        }
      }
    };
    float acc[kNT / 2][4];
    exchange(warp ^ 1, (warp & 1) != 0, o, acc, std::integral_constant<int, kNT / 2>{});
    float fin[kNT / 4][4];
    exchange(warp ^ 2, (warp & 2) != 0, acc, fin, std::integral_constant<int, kNT / 4>{});
    const int col = (warp & 1) * (D / 2) + (warp >> 1) * (D / 4) + 2 * q4;

    // ---- write the row block, or this CTA's part of it ---------------------
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (out_row[i] < 0) continue;
      const bool some = !none[i] && l[i] != 0.f;  // NaN (from NaN or infinite scores) goes through
      const float lb = some ? m[i] + __log2f(l[i]) : NEG_INF;
      if (!some) {
#pragma unroll
        for (int n = 0; n < kNT / 4; ++n) fin[n][2 * i] = fin[n][2 * i + 1] = 0.f;
      }
      const float inv = some ? 1.0f / l[i] : 0.f;
      long long row = out_row[i];
      const int to = S::target(p, w, block, first, g8 + 8 * i, row);
      if (to == 0) {
        uint16_t* const dst = p.out + row * D + col;
#pragma unroll
        for (int n = 0; n < kNT / 4; ++n)
          *reinterpret_cast<uint32_t*>(dst + n * 8) = pack_bf16(fin[n][2 * i] * inv, fin[n][2 * i + 1] * inv);
        if (col == 0) p.lse[row] = lb * 0.69314718055994530942f;
      } else {
        float* const dst = (to == 1 ? p.whole_o[PREFIX] : p.piece_o[PREFIX]) + row * D + col;
#pragma unroll
        for (int n = 0; n < kNT / 4; ++n)
          *reinterpret_cast<float2*>(dst + n * 8) = make_float2(fin[n][2 * i] * inv, fin[n][2 * i + 1] * inv);
        if (col == 0) (to == 1 ? p.whole_l[PREFIX] : p.piece_l[PREFIX])[row] = lb;
      }
    }
    first = false;
  } while (S::next(p, w));
  if (!ok) {  // let every copy in flight land before the CTA's shared memory goes
    for (int i = consumed; i < issued; ++i)
      mbar_wait(bars + 8 * (i % C::kRing), static_cast<uint32_t>(i / C::kRing) & 1u, nullptr);
  }
  paged_end(beside);
}

// BOTH: the first prefix_ctas CTAs take the prefix's shares and the others the
// own keys' (a prefix whose rows of the whole batch fit one block: one launch less,
// 9.0 -> 8.1 us for 4 sequences behind 1000 tokens, 12 heads of 64).  Else the own keys alone.
template <int D, bool BOTH>
__global__ void __launch_bounds__(PagedCfg<D>::kThreads, 2)
    fa_paged_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                    const PagedParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ long long scratch[PagedCfg<D>::kWarps + 2];
  int block = static_cast<int>(blockIdx.x);
  if constexpr (BOTH) {
    if (block < static_cast<int>(p.prefix_ctas)) {
      paged_rows<D, true>(tmK, tmV, p, block, smem_raw, scratch, false);
      return;
    }
    block -= static_cast<int>(p.prefix_ctas);
  }
  paged_rows<D, false>(tmK, tmV, p, block, smem_raw, scratch, !BOTH && p.prefix_len > 0);
}

// ---------------------------------------------------------------------------
// Joins the parts of every row that more than one CTA (or the prefix and the
// own keys) contributed to, and writes the rows that saw no key.
// ---------------------------------------------------------------------------
// Up to so many sequences a warp of the merge sums their units itself, before it
// waits for the parts; of larger batches it reads the plan after the wait.
constexpr int kMergeScan = 256;

// The parts of one row, in order: own keys of CTAs [c0, c1], prefix of [d0, d1].
struct RowParts {
  long long row, c0, x0, d0, y0, units, ctas;
  int n_own, n_all, in_own, in_prefix;  // row inside its row block
  int b, hk, rr;
  __device__ __forceinline__ void locate(const PagedParams& p, long long r) {
    row = r;
    const long long bh = quotient(row, p.rows);
    rr = static_cast<int>(row - bh * p.rows);
    b = static_cast<int>(quotient(bh, p.Hk));
    hk = static_cast<int>(bh - static_cast<long long>(b) * p.Hk);
  }
  // all: units of the launch, u0 and u1: of the sequences before this one, and with it
  __device__ __forceinline__ void find(const PagedParams& p, long long all, long long u0, long long u1) {
    units = all;
    ctas = paged_ctas(p.own_grid, all, least_units(p.rb[0], false));
    const int blocks = row_blocks(p.rows, p.rb[0]);
    const long long each = quotient(u1 - u0, static_cast<long long>(p.Hk) * blocks);
    const long long n = each - extra_units(p.rb[0]);  // tiles; none: each is 0
    x0 = u0 + (static_cast<long long>(hk) * blocks + rr / p.rb[0]) * each;
    in_own = rr % p.rb[0];
    n_own = 0;
    c0 = 0;
    if (n > 0) {
      c0 = cta_of(units, ctas, x0);
      n_own = static_cast<int>(cta_of(units, ctas, x0 + n - 1) - c0) + 1;
    }
    n_all = n_own;
    d0 = y0 = 0;
    in_prefix = 0;
    if (p.prefix_len > 0) {
      const long long pr = static_cast<long long>(b) * p.rows + rr;  // row among the K/V head's prefix rows
      const long long block = quotient(pr, p.rb[1]);
      in_prefix = static_cast<int>(pr - block * p.rb[1]);
      y0 = (static_cast<long long>(hk) * p.prefix_blocks + block) * (p.prefix_tiles + extra_units(p.rb[1]));
      d0 = cta_of(p.prefix_units, p.prefix_ctas, y0);
      n_all += static_cast<int>(cta_of(p.prefix_units, p.prefix_ctas, y0 + p.prefix_tiles - 1) - d0) + 1;
    }
  }
  // Whole warp: locate() done, the rest, and the wait for the parts.  In a small batch everything that does
  // not need them comes before the wait and runs beside the kernel that writes them.  That is the lengths alone,
  // complete before that kernel's CTAs let this one start (each waited first); read from L2, as no wait of this
  // kernel stands between an earlier kernel's lines in this SM's L1 and the load.
  __device__ __forceinline__ void wait(const PagedParams& p) {
    if (p.B <= kMergeScan) {
      const long long per = static_cast<long long>(p.Hk) * row_blocks(p.rows, p.rb[0]);
      const int lane = threadIdx.x & 31;
      long long all = 0, before = 0;
      int mine = 0;
      for (int b0 = 0; b0 < p.B; b0 += 32) {
        unsigned u = 0;  // units of a row block of sequence b0 + lane
        if (b0 + lane < p.B) {
          const SeqKeys s =
              seq_keys(p, __ldcg(p.lens + b0 + lane), p.new_lens ? __ldcg(p.new_lens + b0 + lane) : p.T);
          const int n = tiles_of(s.lo, s.hi, kPagedTile);
          u = n > 0 ? n + extra_units(p.rb[0]) : 0;
        }
        unsigned incl = u;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const unsigned up = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += up;
        }
        // each lane for its own row's sequence
        const int at = min(max(b - b0, 0), 31);
        const unsigned upto = __shfl_sync(0xffffffffu, incl, at), of = __shfl_sync(0xffffffffu, u, at);
        if (b >= b0 && b < b0 + 32) {
          before = all + upto - of;
          mine = static_cast<int>(of);
        }
        all += __shfl_sync(0xffffffffu, incl, 31);
      }
      find(p, all * per, before * per, (before + mine) * per);
      grid_wait();
    } else {
      grid_wait();
      find(p, p.plan[0], p.plan[1 + b], p.plan[2 + b]);
    }
    grid_release();
  }
  // written by the one CTA that held it
  __device__ __forceinline__ bool done(const PagedParams& p) const { return p.prefix_len == 0 && n_own == 1; }
  // O and L of part i
  __device__ __forceinline__ void at(const PagedParams& p, int d, int i, const float*& o, const float*& l) const {
    const int pre = i < n_own ? 0 : 1, k = pre ? i - n_own : i;
    if ((pre ? n_all - n_own : n_own) == 1) {
      o = p.whole_o[pre] + row * d;
      l = p.whole_l[pre] + row;
      return;
    }
    const long long c = (pre ? d0 : c0) + k;
    // piece 0 of a CTA is the row block that holds its first unit, which starts there or before
    const long long first = pre ? cta_start(p.prefix_units, p.prefix_ctas, c) : cta_start(units, ctas, c);
    const long long slot = 2 * c + (first >= (pre ? y0 : x0) ? 0 : 1);
    const long long r = slot * p.rb[pre] + (pre ? in_prefix : in_own);
    o = p.piece_o[pre] + r * d;
    l = p.piece_l[pre] + r;
  }
};

template <int D>
__device__ __forceinline__ void merge_load(const float* src, int lane, float (&v)[D / 32]) {
  if constexpr (D == 128) {
    const float4 t = *reinterpret_cast<const float4*>(src + lane * 4);
    v[0] = t.x; v[1] = t.y; v[2] = t.z; v[3] = t.w;
  } else {
    const float2 t = *reinterpret_cast<const float2*>(src + lane * 2);
    v[0] = t.x; v[1] = t.y;
  }
}
template <int D>
__device__ __forceinline__ void merge_store(const PagedParams& p, long long row, int lane, const float (&acc)[D / 32],
                                            float top, float sum) {
  const float inv = sum != 0.f ? 1.0f / sum : 0.f;  // a NaN among the parts stays one
  uint16_t* const dst = p.out + row * D + lane * (D / 32);
  if constexpr (D == 128)
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv));
  else
    *reinterpret_cast<uint32_t*>(dst) = pack_bf16(acc[0] * inv, acc[1] * inv);
  if (lane == 0) p.lse[row] = sum != 0.f ? (top + __log2f(sum)) * 0.69314718055994530942f : -__int_as_float(0x7f800000);
}

// Few rows, or many parts to a row: WARPS (4 or 2) warps per row take its parts
// in turn, each lane finds one part and its L, and the warps meet in shared
// memory.
template <int D, int WARPS>
__global__ void __launch_bounds__(128) fa_paged_merge_row_kernel(const PagedParams p) {
  constexpr int kPer = D / 32;
  const int warp = (threadIdx.x >> 5) % WARPS, lane = threadIdx.x & 31;  // warp of the row
  const float NEG_INF = -__int_as_float(0x7f800000);
  const long long all = static_cast<long long>(p.B) * p.Hk * p.rows;
  const long long row = static_cast<long long>(blockIdx.x) * (4 / WARPS) + (threadIdx.x >> 5) / WARPS;
  RowParts parts;
  parts.locate(p, min(row, all - 1));
  parts.wait(p);
  const bool idle = row >= all || parts.done(p);
  if (WARPS == 4 && idle) return;
  const int n_all = idle ? 0 : parts.n_all;
  float mx = NEG_INF, sum = 0.f, acc[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
  for (int base = warp; base < n_all; base += 32 * WARPS) {
    const int i = base + lane * WARPS;
    const float* po = nullptr;
    float L = NEG_INF;
    if (i < n_all) {
      const float* pl;
      parts.at(p, D, i, po, pl);
      L = *pl;
    }
    const int count = min(32, (n_all - base + WARPS - 1) / WARPS);
    auto src = [&](int k) -> const float* {
      return reinterpret_cast<const float*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(po), k));
    };
    // the first part's O travels beside the Ls
    float v0[kPer];
    merge_load<D>(src(0), lane, v0);
    float top = fmaxf(mx, L);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float a = mx == NEG_INF ? 0.f : ex2(mx - top);  // no key in any part: every weight is 0
    const float wt = L == NEG_INF ? 0.f : ex2(L - top);
    float ws = wt;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ws += __shfl_xor_sync(0xffffffffu, ws, o);
    mx = top;
    sum = a * sum + ws;
    const float w0 = __shfl_sync(0xffffffffu, wt, 0);
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] = a * acc[e] + w0 * v0[e];
#pragma unroll 4
    for (int k = 1; k < count; ++k) {
      float v[kPer];
      merge_load<D>(src(k), lane, v);
      const float c = __shfl_sync(0xffffffffu, wt, k);
#pragma unroll
      for (int e = 0; e < kPer; ++e) acc[e] = fmaf(c, v[e], acc[e]);
    }
  }
  __shared__ float shared[4][D + 2];
  float (*const sh)[D + 2] = shared + (threadIdx.x >> 5) / WARPS * WARPS;  // the row's warps
#pragma unroll
  for (int e = 0; e < kPer; ++e) sh[warp][lane * kPer + e] = acc[e];
  if (lane == 0) {
    sh[warp][D] = mx;
    sh[warp][D + 1] = sum;
  }
  __syncthreads();
  if (warp != 0 || idle) return;
  float top = NEG_INF;
#pragma unroll
  for (int i = 0; i < WARPS; ++i) top = fmaxf(top, sh[i][D]);
  sum = 0.f;
#pragma unroll
  for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
#pragma unroll
  for (int i = 0; i < WARPS; ++i) {
    // a warp whose parts hold no key, or nothing but NaN, has top -inf: its sum counts as it is
    const float c = sh[i][D] == NEG_INF ? 1.f : ex2(sh[i][D] - top);
    sum += c * sh[i][D + 1];
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] += c * sh[i][lane * kPer + e];
  }
  merge_store<D>(p, parts.row, lane, acc, top, sum);
}

// Many rows: one warp joins four of them at once.  Eight lanes find the parts
// and Ls of each row, then the whole warp sums O row by row with D / 32 columns
// to a lane, the four rows' loads in flight together.
template <int D>
__global__ void __launch_bounds__(128) fa_paged_merge_rows_kernel(const PagedParams p) {
  constexpr int kPer = D / 32, kRows = 4;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float NEG_INF = -__int_as_float(0x7f800000);
  const long long all = static_cast<long long>(p.B) * p.Hk * p.rows;
  const long long row0 = (static_cast<long long>(blockIdx.x) * 4 + warp) * kRows;
  const int group = lane >> 3;
  RowParts parts;
  parts.locate(p, min(row0 + group, all - 1));
  parts.wait(p);
  if (row0 >= all) return;
  const int n_mine = (row0 + group < all && !parts.done(p)) ? parts.n_all : 0;
  const bool write = row0 + group < all && !parts.done(p);
  const int most = __reduce_max_sync(0xffffffffu, static_cast<unsigned>(n_mine));
  float mx = NEG_INF, sum = 0.f;  // of this lane's row
  float acc[kRows][kPer];
#pragma unroll
  for (int r = 0; r < kRows; ++r)
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[r][e] = 0.f;
  for (int base = 0; base < most; base += 8) {
    const int i = base + (lane & 7);
    const float* po = nullptr;  // no part, or one without a key that the row sees
    float L = NEG_INF;
    if (i < n_mine) {
      const float* pl;
      parts.at(p, D, i, po, pl);
      L = *pl;
      if (L == NEG_INF) po = nullptr;
    }
    float top = fmaxf(mx, L);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float a = mx == NEG_INF ? 0.f : ex2(mx - top);
    const float wt = L == NEG_INF ? 0.f : ex2(L - top);
    float ws = wt;
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) ws += __shfl_xor_sync(0xffffffffu, ws, o);
    mx = top;
    sum = a * sum + ws;
    if (base > 0) {
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const float ar = __shfl_sync(0xffffffffu, a, r * 8);
#pragma unroll
        for (int e = 0; e < kPer; ++e) acc[r][e] *= ar;
      }
    }
    const int count = min(8, most - base);
#pragma unroll 2
    for (int k = 0; k < count; ++k) {
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const float c = __shfl_sync(0xffffffffu, wt, r * 8 + k);
        const float* const src = reinterpret_cast<const float*>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(po), r * 8 + k));
        if (src != nullptr) {  // a weight of zero multiplies all the same: 0 * NaN is NaN
          float v[kPer];
          merge_load<D>(src, lane, v);
#pragma unroll
          for (int e = 0; e < kPer; ++e) acc[r][e] = fmaf(c, v[e], acc[r][e]);
        }
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const float top = __shfl_sync(0xffffffffu, mx, r * 8), tot = __shfl_sync(0xffffffffu, sum, r * 8);
    if (__shfl_sync(0xffffffffu, static_cast<int>(write), r * 8)) merge_store<D>(p, row0 + r, lane, acc[r], top, tot);
  }
}

}  // namespace fa
