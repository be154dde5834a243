// fa_paged.cu -- entry points of attention over the paged cache: fa_fwd_paged,
// fa_fwd_prefix and their workspace size.  See include/fa.h for their contracts.
#include <atomic>
#include <cmath>
#include <cstdint>

#include "fa.h"
#include "fa_host.h"
#include "fa_paged_kernel.cuh"
#include "fa_paged_tile.cuh"

namespace {

constexpr int kMaxKeys = 1 << 30;  // tokens of a sequence or a prefix: tile arithmetic stays within an int

std::atomic<bool> g_ready[fa_host::kMaxDevices];

template <typename K>
bool allow(K kernel, size_t smem) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) ==
         cudaSuccess;
}

// The tile kernels move registers between warpgroups, which assumes the count
// they are launched with; a build with another count is refused.
template <int D, bool PREFIX, bool PAIR>
bool allow_tile() {
  using C = fa::TileCfg<D, PAIR>;
  cudaFuncAttributes a;
  return cudaFuncGetAttributes(&a, fa::fa_paged_tile_kernel<D, PREFIX, PAIR>) == cudaSuccess &&
         a.numRegs == C::kRegLaunch && allow(fa::fa_paged_tile_kernel<D, PREFIX, PAIR>, C::kSmemBytes);
}

template <int D>
bool opt_in() {
  return allow(fa::fa_paged_kernel<D, false>, fa::PagedCfg<D>::kSmemBytes) &&
         allow(fa::fa_paged_kernel<D, true>, fa::PagedCfg<D>::kSmemBytes) && allow_tile<D, false, false>() &&
         allow_tile<D, false, true>() && allow_tile<D, true, false>() && allow_tile<D, true, true>();
}

// The kernels' shared-memory opt-in, once per device (a repeated call is harmless).
int ready(int dev) {
  if (g_ready[dev].load(std::memory_order_acquire)) return FA_OK;
  if (!opt_in<64>() || !opt_in<128>()) return FA_ERR_LAUNCH;
  g_ready[dev].store(true, std::memory_order_release);
  return FA_OK;
}

using fa_host::make_cache_map;

size_t up(size_t n) { return (n + 255) / 256 * 256; }

// Rows per row block, by the rows that share each K/V byte: the warp-level
// kernel's 16, or the tcgen05 kernel's 128 (one query tile) or 256 (a pair).
// d = 128, 16 sequences x 8192 keys, 2 K/V heads, us: 16 rows 29.5 on the
// warp-level kernel, 35.9 on the tile kernel (1000 keys: 11.1, 14.9); 32 rows as
// two row blocks of 16 read K and V twice, 33.2 against 36.6 while they stay in
// L2, but 319 against 169 for 32 x 8192 keys of 8 heads; blocks of 32 rows on
// warp-level MMAs run at 158 TFLOP/s, that path's rate: 16 x up to 1000 keys 12.8
// against 15.6, but 32 x up to 8192 of 8 heads 113.8 against 103.2, and the host
// does not know the lengths; 128 rows 41.9 on one
// query tile, 44.8 as half of a pair; 256 rows 47.8 on a pair, 52.6 on two tiles.
int block_rows(long long rows) { return rows <= 16 ? 16 : (rows <= 128 ? 128 : 256); }
constexpr int kTileKeys = fa::kPagedTile;
// A wave of one kind's CTAs.  (With a prefix that takes most SMs, own keys run in a second wave; no CTA waits for
// another but at its end, for a grid that has started whole.)
int grid_of(int block_rows, int sms) { return block_rows == 16 ? 2 * sms : sms; }

// The row blocks, tiles and CTAs of a call, and the parts of its workspace, in
// order; every part begins on a 256-byte boundary.
struct Layout {
  int rb[2], grid[2];
  int prefix_blocks, prefix_tiles;
  long long prefix_units, prefix_ctas;
  size_t plan, piece_o[2], piece_l[2], whole_o[2], whole_l[2];
  size_t bytes() const {
    size_t n = plan + 240;  // the caller aligns the workspace to 16 bytes, its parts to 256
    for (int i = 0; i < 2; ++i) n += piece_o[i] + piece_l[i] + whole_o[i] + whole_l[i];
    return n;
  }
};
Layout layout(int B, int H, int Hk, int T, int d, int prefix_len, int sms) {
  const size_t all = static_cast<size_t>(B) * H * T;
  const long long rows = static_cast<long long>(H / Hk) * T;
  Layout l = {};
  l.plan = up((static_cast<size_t>(B) + 3) * sizeof(long long));
  for (int i = 0; i < (prefix_len > 0 ? 2 : 1); ++i) {
    l.rb[i] = block_rows(i == 0 ? rows : rows * B);
    l.grid[i] = grid_of(l.rb[i], sms);
    if (i == 1) {
      l.prefix_blocks = fa::row_blocks(rows * B, l.rb[1]);
      l.prefix_tiles = (prefix_len + kTileKeys - 1) / kTileKeys;
      l.prefix_units = 1ll * Hk * l.prefix_blocks * (l.prefix_tiles + fa::extra_units(l.rb[1]));
      l.prefix_ctas = fa::paged_ctas(l.grid[1], l.prefix_units, fa::least_units(l.rb[1], true));
      l.grid[1] = static_cast<int>(l.prefix_ctas);
    }
    const size_t pieces = 2 * static_cast<size_t>(l.grid[i]) * l.rb[i];
    l.piece_o[i] = up(pieces * d * sizeof(float));
    l.piece_l[i] = up(pieces * sizeof(float));
    l.whole_o[i] = prefix_len > 0 ? up(all * d * sizeof(float)) : 0;
    l.whole_l[i] = prefix_len > 0 ? up(all * sizeof(float)) : 0;
  }
  return l;
}

// The merge: one warp joins four rows where rows are many for their parts (it takes the parts of its rows one
// after another: from kMergeRows rows and kMergeRowsPerPart times the parts of a row), else two warps join one row
// (from kMergeTwo rows: the four-warp form's CTAs come in waves then) or four do.  Whole calls, us, with a warp for
// four rows / two to one / four to one:
//   rows of parts: 16000 of 3: 45.7 / 65.2 / 83.8;  7680 of 6: 32.8 / 38.0 / 46.6;  6144 of 7 (d = 64): 24.6 / 26.1 /
//   33.8;  5120 of 4: 25.6 / 28.2 / 33.4;  4096 of 5: 23.6 / 24.8 / 28.9;  2560 of 2: 20.4 / 21.5 / 23.2
//   the other side: 5120 of 8: 33.5 / 32.4 / 37.8;  4096 of 10: 30.6 / 28.0 / 32.3;  2560 of 8: 22.3 / 21.0 / 22.9;
//   2048 of 20: 31.1 / 22.7 / 27.6;  1920 of 2: 26.4 / 25.5 / 28.3;  1600 of 4: 25.4 / 22.4 / 26.2
//   few rows: 1280 of 4: 19.9 / 17.1 / 18.2;  1024 of 5: 21.6 / 17.8 / 18.6;  1024 of 39: 26.3 / 21.4 / 21.2;  768 of 26:
//   19.8 / 17.1 / 16.8;  512 of 3: 25.9 / 23.7 / 23.6;  160 of 31: 21.6 / 11.4 / 10.6;  16 of 77: 23.2 / 9.9 / 9.3
constexpr long long kMergeRows = 2400, kMergeRowsPerPart = 700, kMergeTwo = 1024;

using fa_host::launch_kernel;

template <int D>
int launch_merge(const fa::PagedParams& p, long long rows, cudaStream_t stream) {
  // parts of a row where the shares cut every row block alike
  long long parts = p.own_grid / (1ll * p.B * p.Hk * fa::row_blocks(p.rows, p.rb[0])) + 1;
  if (p.prefix_len > 0) parts += p.prefix_ctas / (1ll * p.Hk * p.prefix_blocks) + 1;
  if (rows >= kMergeRows && rows >= kMergeRowsPerPart * parts)
    return launch_kernel(fa::fa_paged_merge_rows_kernel<D>, (rows + 15) / 16, 128, 0, stream, p);
  if (rows >= kMergeTwo)
    return launch_kernel(fa::fa_paged_merge_row_kernel<D, 2>, (rows + 1) / 2, 128, 0, stream, p);
  return launch_kernel(fa::fa_paged_merge_row_kernel<D, 4>, rows, 128, 0, stream, p);
}

struct Caches {
  const void *k, *v;
  const long long* strides;
  int d, page, Hk, n_pages;
  bool maps(CUtensorMap* mk, CUtensorMap* mv, int box_rows) const {
    const int rows = box_rows < page ? box_rows : page;
    return make_cache_map(mk, k, d, page, Hk, n_pages, strides, rows) &&
           make_cache_map(mv, v, d, page, Hk, n_pages, strides + 3, rows);
  }
};

// One part of a call: the prefix or the sequences' own keys.
template <int D, bool PREFIX>
int launch_part(const Caches& c, const fa::PagedParams& p, int grid, cudaStream_t stream) {
  const int rb = p.rb[PREFIX];  // a prefix's is 128 or 256 here
  CUtensorMap mk, mv;
  if (!c.maps(&mk, &mv, rb == 16 ? fa::PagedCfg<D>::kKeys : kTileKeys)) return FA_ERR_LAUNCH;
  if (!PREFIX && rb == 16) {
    using S = fa::PagedCfg<D>;
    return launch_kernel(fa::fa_paged_kernel<D, false>, grid, S::kThreads, S::kSmemBytes, stream, mk, mv, p);
  }
  if (rb == 128) {
    using T = fa::TileCfg<D, false>;
    return launch_kernel(fa::fa_paged_tile_kernel<D, PREFIX, false>, grid, T::kThreads, T::kSmemBytes, stream, mk, mv,
                         p);
  }
  using T = fa::TileCfg<D, true>;
  return launch_kernel(fa::fa_paged_tile_kernel<D, PREFIX, true>, grid, T::kThreads, T::kSmemBytes, stream, mk, mv, p);
}

template <int D>
int launch(const Caches& c, const fa::PagedParams& p, const Layout& l, long long rows, cudaStream_t stream) {
  int st = FA_OK;
  if (p.prefix_len > 0 && l.rb[1] == 16) {  // and so l.rb[0] == 16
    using S = fa::PagedCfg<D>;
    CUtensorMap mk, mv;
    if (!c.maps(&mk, &mv, S::kKeys)) return FA_ERR_LAUNCH;
    st = launch_kernel(fa::fa_paged_kernel<D, true>, p.prefix_ctas + p.own_grid, S::kThreads, S::kSmemBytes, stream,
                       mk, mv, p);
  } else {
    if (p.prefix_len > 0) st = launch_part<D, true>(c, p, l.grid[1], stream);
    if (st == FA_OK) st = launch_part<D, false>(c, p, p.own_grid, stream);
  }
  return st == FA_OK ? launch_merge<D>(p, rows, stream) : st;
}

int paged_impl(const void* q, const void* k_cache, const void* v_cache, void* o, float* lse, const int* prefix_pages,
               int prefix_len, const int* block_table, const int* seq_lens, const int* new_lens,
               const long long* strides, int B, int H, int Hk, int T, int d, int n_pages, int page_size, int max_pages,
               float scale, int left, int right, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  const bool noop = T == 0;
  if (!k_cache || !v_cache || !block_table || !seq_lens || !strides || (prefix_len > 0 && !prefix_pages) ||
      (!noop && (!q || !o || !lse || !workspace)))
    return FA_ERR_NULL;
  const void* big[] = {q, k_cache, v_cache, o, lse, workspace};
  for (const void* x : big)
    if (reinterpret_cast<uintptr_t>(x) & 15u) return FA_ERR_ALIGN;
  if ((reinterpret_cast<uintptr_t>(block_table) | reinterpret_cast<uintptr_t>(seq_lens) |
       reinterpret_cast<uintptr_t>(new_lens) | reinterpret_cast<uintptr_t>(prefix_pages)) & 3u)
    return FA_ERR_ALIGN;
  if (d != 64 && d != 128) return FA_ERR_HEADDIM;
  if (B <= 0 || H <= 0 || Hk <= 0 || T < 0 || H % Hk != 0) return FA_ERR_SHAPE;
  if (n_pages <= 0 || max_pages <= 0 || page_size < 16 || page_size > 256 || (page_size & (page_size - 1)))
    return FA_ERR_SHAPE;
  if (left < -1 || right < -1 || prefix_len < 0 || prefix_len > kMaxKeys) return FA_ERR_SHAPE;
  const long long rows = static_cast<long long>(B) * H * T;
  if (static_cast<long long>(max_pages) * page_size > kMaxKeys || static_cast<long long>(B) * H >= (1ll << 31) ||
      rows >= (1ll << 31) - 256)  // a row block's last row still has an int's index
    return FA_ERR_SHAPE;
  if (!std::isfinite(scale) || !(scale > 0.f)) return FA_ERR_SCALE;
  for (int i = 0; i < 6; ++i)  // page, head and token strides of K, then of V; a tensor map's limit is 2^40 bytes
    if (strides[i] < 8 || (strides[i] & 7) || strides[i] >= (1ll << 39)) return FA_ERR_STRIDE;
  if (noop) return FA_OK;
  int dev = -1, sms = 0;
  int st = fa_host::current_device(&dev, &sms);
  if (st != FA_OK) return st;
  const Layout l = layout(B, H, Hk, T, d, prefix_len, sms);
  if (workspace_bytes < l.bytes()) return FA_ERR_WORKSPACE;
  const void* ptrs[] = {q, k_cache, v_cache, o, lse, workspace, block_table, seq_lens};
  for (const void* x : ptrs)
    if (!fa_host::is_device_pointer(x, dev)) return FA_ERR_POINTER;
  if ((new_lens && !fa_host::is_device_pointer(new_lens, dev)) ||
      (prefix_len > 0 && !fa_host::is_device_pointer(prefix_pages, dev)))
    return FA_ERR_POINTER;
  st = ready(dev);
  if (st != FA_OK) return st;
  fa::PagedParams p = {};
  p.q = static_cast<const uint16_t*>(q);
  p.out = static_cast<uint16_t*>(o);
  p.lse = lse;
  p.table = block_table;
  p.lens = seq_lens;
  p.new_lens = new_lens;
  p.prefix_pages = prefix_pages;
  p.B = B;
  p.Hk = Hk;
  p.T = T;
  p.rows = H / Hk * T;
  p.n_pages = n_pages;
  p.max_pages = max_pages;
  while ((1 << p.page_shift) < page_size) ++p.page_shift;
  p.capacity = max_pages * page_size;
  p.prefix_len = prefix_len;
  p.left = left;
  p.right = right;
  p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634074);
  p.rb[0] = l.rb[0];
  p.rb[1] = l.rb[1];
  p.prefix_blocks = l.prefix_blocks;
  p.prefix_tiles = l.prefix_tiles;
  p.prefix_units = l.prefix_units;
  p.prefix_ctas = l.prefix_ctas;
  char* at = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(workspace) + 255) & ~static_cast<uintptr_t>(255));
  p.plan = reinterpret_cast<long long*>(at);
  at += l.plan;
  for (int i = 0; i < 2; ++i) {
    p.piece_o[i] = reinterpret_cast<float*>(at);
    p.piece_l[i] = reinterpret_cast<float*>(at += l.piece_o[i]);
    p.whole_o[i] = reinterpret_cast<float*>(at += l.piece_l[i]);
    p.whole_l[i] = reinterpret_cast<float*>(at += l.whole_o[i]);
    at += l.whole_l[i];
  }
  p.status = fa_host::status_word(dev);
  if (!p.status) return FA_ERR_LAUNCH;
  // Beside a prefix that leaves a quarter of the SMs or more free, the own keys are cut for the free ones alone: a
  // share that has to wait for a prefix CTA's SM ends last, whatever the lengths.  us, cut for the free SMs / for
  // all: 16 sequences behind 2000 tokens (prefix on 40 of 152 SMs), up to 100 own keys 19.0 / 20.2, 1000 23.0 / 26.6,
  // 4000 34.9 / 45.4, 30000 159 / 167;  64 behind 500 (8), 4000 own 94.9 / 118;  100 behind 6000 (51), 60 own
  // 31.0 / 33.1;  12 x 2 tokens behind 5800 (100), 300 own 18.5 / 22.0;  behind 6300 (108), 3000 own 37.2 / 36.4;  the
  // worst: 40 x 2 behind 12000 (49), 200 own 29.7 / 28.3.  Past three quarters: behind 7200 (122), 300 own
  // 19.7 / 22.9, 3000 own 46.1 / 37.7;  30 x 20 tokens behind 3000 (133), 900 own 62.2 / 48.3.
  // (Prefix rows in one block of 16: two CTAs of that launch fit an SM, but own keys cut for all free places are
  // slower, 9.3 for 8.1 with 4 sequences behind 1000 tokens, 12 heads of 64.)
  p.own_grid = l.grid[0];
  if (prefix_len > 0 && l.prefix_ctas * 4 <= 3ll * sms)
    p.own_grid = p.own_grid / sms * static_cast<int>(sms - l.prefix_ctas);
  const Caches c = {k_cache, v_cache, strides, d, page_size, Hk, n_pages};
  return d == 64 ? launch<64>(c, p, l, rows, stream) : launch<128>(c, p, l, rows, stream);
}

}  // namespace

extern "C" {

size_t fa_paged_workspace_bytes(int B, int H, int Hk, int T, int d, int prefix_len) {
  if (B <= 0 || H <= 0 || Hk <= 0 || H % Hk != 0 || T <= 0 || (d != 64 && d != 128) || prefix_len < 0 ||
      prefix_len > kMaxKeys)
    return 0;
  int dev = -1, sms = 0;
  if (fa_host::current_device(&dev, &sms) != FA_OK) sms = 148;
  return layout(B, H, Hk, T, d, prefix_len, sms).bytes();
}

int fa_fwd_paged(const void* q, const void* k_cache, const void* v_cache, void* o, float* lse, const int* block_table,
                 const int* seq_lens, const int* new_lens, const long long* strides, int B, int H, int Hk, int T, int d,
                 int n_pages, int page_size, int max_pages, float scale, int window_left, int window_right,
                 void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  return paged_impl(q, k_cache, v_cache, o, lse, nullptr, 0, block_table, seq_lens, new_lens, strides, B, H, Hk, T, d,
                    n_pages, page_size, max_pages, scale, window_left, window_right, workspace, workspace_bytes,
                    stream);
}

int fa_fwd_prefix(const void* q, const void* k_cache, const void* v_cache, void* o, float* lse,
                  const int* prefix_pages, int prefix_len, const int* block_table, const int* seq_lens,
                  const int* new_lens, const long long* strides, int B, int H, int Hk, int T, int d, int n_pages,
                  int page_size, int max_pages, float scale, void* workspace, size_t workspace_bytes,
                  cudaStream_t stream) {
  if (prefix_len <= 0) return FA_ERR_SHAPE;
  return paged_impl(q, k_cache, v_cache, o, lse, prefix_pages, prefix_len, block_table, seq_lens, new_lens, strides, B,
                    H, Hk, T, d, n_pages, page_size, max_pages, scale, -1, 0, workspace, workspace_bytes, stream);
}

}  // extern "C"
