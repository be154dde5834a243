// fa_cache.cu -- entry points that keep a paged cache small: fa_kv_weights and
// fa_kv_evict with its workspace size.  See include/fa.h for their contracts.
#include <atomic>
#include <cmath>
#include <cstdint>

#include "fa.h"
#include "fa_evict_kernel.cuh"
#include "fa_host.h"
#include "fa_weights_kernel.cuh"

namespace {

constexpr int kMaxKeys = 1 << 30;  // tokens of a sequence: tile arithmetic stays within an int

bool misaligned(const void* p, unsigned bytes) { return reinterpret_cast<uintptr_t>(p) & (bytes - 1); }

// Strides of bf16 views in multiples of 16 bytes, and of the weights (any).
bool stride_ok(long long s, int multiple) { return s >= multiple && s % multiple == 0 && s < (1ll << 39); }

int page_shift_of(int page_size) {
  int s = 0;
  while ((1 << s) < page_size) ++s;
  return s;
}
bool page_sizes_ok(int n_pages, int page_size, int max_pages) {
  return n_pages > 0 && max_pages > 0 && page_size >= 16 && page_size <= 256 && (page_size & (page_size - 1)) == 0 &&
         static_cast<long long>(max_pages) * page_size <= kMaxKeys;
}

// 3-D map over the queries: (d, row of [B * H * T], 1), 128-byte swizzle, `box_rows` rows x 64 elements per box.
bool make_rows_map(CUtensorMap* map, const void* ptr, int d, long long rows, int box_rows) {
  fa_host::EncodeTiledFn enc = fa_host::encode_fn();
  if (!enc) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(rows), 1u};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2u, static_cast<cuuint64_t>(rows) * d * 2u};
  cuuint32_t box[3] = {64u, static_cast<cuuint32_t>(box_rows), 1u};
  cuuint32_t estr[3] = {1u, 1u, 1u};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

std::atomic<bool> g_ready[fa_host::kMaxDevices];

template <typename K>
bool allow(K kernel, size_t smem) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) ==
         cudaSuccess;
}

// Weights that a CTA of the selection holds: as many as fit beside its histogram; up to kSelectSmall 512 threads do.
constexpr int kSelectWindow = 48 << 10, kSelectSmall = 4 << 10;

// The kernels' shared-memory opt-in, once per device (a repeated call is harmless).
int ready(int dev) {
  if (g_ready[dev].load(std::memory_order_acquire)) return FA_OK;
  if (!allow(fa::fa_kv_weights_tile_kernel<64>, fa::WTileCfg<64>::kSmemBytes) ||
      !allow(fa::fa_kv_weights_tile_kernel<128>, fa::WTileCfg<128>::kSmemBytes) ||
      !allow(fa::fa_evict_select_kernel<512>, kSelectSmall * sizeof(float)) ||
      !allow(fa::fa_evict_select_kernel<1024>, kSelectWindow * sizeof(float)) ||
      !allow(fa::fa_evict_list_kernel, kSelectWindow * sizeof(float)))
    return FA_ERR_LAUNCH;
  g_ready[dev].store(true, std::memory_order_release);
  return FA_OK;
}

// fa_host::launch_kernel for a grid of clusters.
template <typename K, typename... A>
int launch_clusters(K kernel, long long clusters, int cluster, int threads, size_t smem, cudaStream_t stream,
                    const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * cluster));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return fa_host::launched(cudaLaunchKernelEx(&cfg, kernel, args...));
}

// Rows of a (sequence, K/V head) up to which the warp-level kernel takes them.  us on it / on the tensor cores, 16
// sequences x 8192 keys, 8 K/V heads of 128: 16 rows 59 / 141, 32 83 / 141, 48 110 / 142, 64 138 / 141, 96 193 / 142;  8 x
// 1000 keys, 2 heads: 16 rows 5.4 / 7.6, 32 6.9 / 7.6, 48 8.3 / 7.6, 64 9.8 / 7.6;  d = 64 within 5% of these.
constexpr int kWarpRows = 48;

template <int D>
int launch_weights(fa::WeightsParams& p, long long all_rows, int page_size, int sms, cudaStream_t stream) {
  if (p.s.rows <= kWarpRows) {
    // 8 KB of K to a warp, or where those units are fewer than the places (by the table's width) 4 KB
    constexpr int kM = 256 / D;
    const long long grid = 3ll * sms;
    const int tile = fa::WRowsCfg<kM>::kTile;
    if (1ll * p.s.B * p.s.Hk * ((p.s.capacity + tile - 1) / tile) >= grid)
      return fa_host::launch_kernel(fa::fa_kv_weights_kernel<D, kM>, grid, fa::kWeightThreads, 0, stream, p);
    return fa_host::launch_kernel(fa::fa_kv_weights_kernel<D, kM / 2>, grid, fa::kWeightThreads, 0, stream, p);
  }
  using C = fa::WTileCfg<D>;
  CUtensorMap mk, mq;
  const long long strides[3] = {p.k_page, p.k_head, p.k_token};
  if (!fa_host::make_cache_map(&mk, p.k, D, page_size, p.s.Hk, p.s.n_pages, strides,
                               page_size < fa::kWeightTile ? page_size : fa::kWeightTile) ||
      !make_rows_map(&mq, p.s.q, D, all_rows, C::kPiece))
    return FA_ERR_LAUNCH;
  // CTAs to a unit: two where a unit has many row blocks (us with 1 / 2 / 4, 32/8 heads of 128: 4096 tokens over 8192
  // keys 229 / 215 / 268, 2 x 2048 over 8192 231 / 204 / 352, 8 x 512 over 4096 129 / 121 / 290; 12 heads, 8 x 1024 over
  // 1024, 8 blocks: 34.6 / 35.2 / 63.5), and two or four where even they leave SMs without a unit (1024 over 1024:
  // 38.5 / 23.4 / 17.1;  8/2 heads, 4096 over 4096: 119 / 64 / 38;  12 heads, 1024 over 1024: 14.2 / 11.6 / 16.8).  Clusters of
  // four do not fill all SMs, which the wide ones of the first lines pay for.
  const int blocks = (p.s.rows + 127) / 128;
  const long long units = 1ll * p.s.B * p.s.Hk * ((p.s.capacity + C::kUnit - 1) / C::kUnit);  // at most
  int cluster = blocks >= 16 ? 2 : 1;
  if (blocks >= 4 && 4 * units <= sms) cluster = 4;
  else if (blocks >= 2 && 2 * units <= sms) cluster = 2;
  long long grid = sms / cluster;
  if (grid > units) grid = units;
  // units that a CTA works long on are given out one by one: by the number of clusters, and by the rows, which the lengths
  // on the device may yet leave too few of
  p.uneven = blocks >= 20 * cluster && grid <= 32 * fa::WTileUnits::kMost;
  return launch_clusters(fa::fa_kv_weights_tile_kernel<D>, grid, cluster, C::kThreads, C::kSmemBytes, stream, mk, mq, p);
}

// CTAs to a head's K or V, while each has rows to move: in place a cluster of at most 8, up to three CTAs per SM in all
// (16 x up to 8192 keys halved, 128 heads, the move alone with 1 / 2 / 4 / 8: 100 / 76 / 76 / 83 us); into other pages,
// where none waits for another, up to four (4 x up to 31999 to 8000, 16 heads: 162 / 92 / 55 / 35 us).
template <int D>
int launch_move(fa::EvictParams& p, long long heads, int sms, cudaStream_t stream) {
  constexpr int kRound = fa::kMoveThreads / (D / 8) * 8;  // rows of a CTA and round
  const bool fork = p.table_out != p.table;
  p.parts = 1;
  while (p.parts < (fork ? 64 : 8) && 2 * heads * p.parts < (fork ? 4ll : 3ll) * sms &&
         static_cast<long long>(kRound) * p.parts < p.most)
    p.parts *= 2;
  if (fork)
    return fa_host::launch_kernel(fa::fa_evict_move_kernel<D>, 3 * heads * p.parts, fa::kMoveThreads, 0, stream, p);
  return launch_clusters(fa::fa_evict_move_kernel<D>, 3 * heads, p.parts, fa::kMoveThreads, 0, stream, p);
}

// The workspace: what the selection leaves per head, then what its parts leave for one another.
// From how many weights of a head (the capacity, times what of it leaves a CTA) the selection goes in parts.  The whole
// call, into other pages, us with one CTA to a head / in parts: 16384 tokens, 1 head 25 / 26, 16 heads 34 / 39; 32768: 1 head
// 38 / 27, 8 46 / 42, 16 64 / 60, 32 91 / 93; 65536: 8 heads 109 / 63, 32 197 / 181, 64 327 / 314; 131072: 1 head 151 / 35.
constexpr long long kSplitWeights = 26 << 10;

struct EvictWorkspace {
  size_t found, above, hist, bytes;  // offsets of 16 bytes
  EvictWorkspace(int B, int Hk) {
    const size_t heads = static_cast<size_t>(B) * Hk, parts = fa::select_parts(static_cast<long long>(heads));
    found = heads * sizeof(fa::EvictHead);
    bytes = above = hist = found;
    if (parts < 2) return;
    above = found + 2 * heads * sizeof(fa::EvictFound);
    hist = above + (heads * parts * sizeof(int) + 15) / 16 * 16;
    bytes = hist + 2 * heads * parts * fa::kSelectBins * sizeof(int);
  }
};

int launch_select(fa::EvictParams& p, const EvictWorkspace& at, long long heads, cudaStream_t stream) {
  const int parts = fa::select_parts(heads);
  if (parts >= 2 && p.capacity * (parts - 1ll) >= kSplitWeights * parts) {
    uint8_t* const ws = reinterpret_cast<uint8_t*>(p.heads);
    p.found = reinterpret_cast<fa::EvictFound*>(ws + at.found);
    p.above = reinterpret_cast<int*>(ws + at.above);
    p.hist = reinterpret_cast<int*>(ws + at.hist);
    p.split = parts;
    const int part = (p.capacity / parts + 511) & ~255;  // of the longest sequence, not less
    p.window = part < kSelectWindow ? part : kSelectWindow;
    const long long grid = heads * parts;
    constexpr int kT = fa::kSplitThreads;
    int st = fa_host::launch_kernel(fa::fa_evict_count_kernel<0>, grid, kT, 0, stream, p);
    if (st == FA_OK) st = fa_host::launch_kernel(fa::fa_evict_count_kernel<1>, grid, kT, 0, stream, p);
    if (st == FA_OK) st = fa_host::launch_kernel(fa::fa_evict_count_kernel<2>, grid, kT, 0, stream, p);
    if (st == FA_OK)
      st = fa_host::launch_kernel(fa::fa_evict_list_kernel, grid, kT, p.window * sizeof(float), stream, p);
    return st;
  }
  p.window = p.capacity < kSelectWindow ? p.capacity : kSelectWindow;
  const size_t smem = p.window * sizeof(float);
  return p.window <= kSelectSmall ? fa_host::launch_kernel(fa::fa_evict_select_kernel<512>, heads, 512, smem, stream, p)
                                  : fa_host::launch_kernel(fa::fa_evict_select_kernel<1024>, heads, 1024, smem, stream, p);
}

}  // namespace

extern "C" {

int fa_kv_weights(const void* q, const float* lse, const void* k_cache, float* weights, const int* block_table,
                  const int* seq_lens, const int* new_lens, const long long* strides, int B, int H, int Hk, int T, int d,
                  int n_pages, int page_size, int max_pages, float scale, int window_left, int window_right,
                  float decay, cudaStream_t stream) {
  const bool noop = T == 0;
  if (!k_cache || !weights || !block_table || !seq_lens || !strides || (!noop && (!q || !lse))) return FA_ERR_NULL;
  if (misaligned(q, 16) || misaligned(k_cache, 16) || misaligned(lse, 4) || misaligned(weights, 4) ||
      misaligned(block_table, 4) || misaligned(seq_lens, 4) || misaligned(new_lens, 4))
    return FA_ERR_ALIGN;
  if (d != 64 && d != 128) return FA_ERR_HEADDIM;
  if (B <= 0 || H <= 0 || Hk <= 0 || T < 0 || H % Hk != 0 || !page_sizes_ok(n_pages, page_size, max_pages))
    return FA_ERR_SHAPE;
  if (window_left < -1 || window_right < -1) return FA_ERR_SHAPE;
  if (static_cast<long long>(B) * H >= (1ll << 31) || static_cast<long long>(B) * H * T >= (1ll << 31) - 256)
    return FA_ERR_SHAPE;
  if (!std::isfinite(scale) || !(scale > 0.f)) return FA_ERR_SCALE;
  if (!std::isfinite(decay) || !(decay >= 0.f)) return FA_ERR_SCALE;
  for (int i = 0; i < 5; ++i)  // page, head and token strides of K; page and head strides of the weights
    if (!stride_ok(strides[i], i < 3 ? 8 : 1)) return FA_ERR_STRIDE;
  if (noop) return FA_OK;
  int dev = -1, sms = 0;
  const int st = fa_host::current_device(&dev, &sms);
  if (st != FA_OK) return st;
  const void* ptrs[] = {q, lse, k_cache, weights, block_table, seq_lens};
  for (const void* x : ptrs)
    if (!fa_host::is_device_pointer(x, dev)) return FA_ERR_POINTER;
  if (new_lens && !fa_host::is_device_pointer(new_lens, dev)) return FA_ERR_POINTER;
  if (const int r = ready(dev); r != FA_OK) return r;
  fa::WeightsParams p = {};
  p.s.q = static_cast<const uint16_t*>(q);
  p.s.lse = const_cast<float*>(lse);
  p.s.table = block_table;
  p.s.lens = seq_lens;
  p.s.new_lens = new_lens;
  p.s.B = B;
  p.s.Hk = Hk;
  p.s.T = T;
  p.s.rows = H / Hk * T;
  p.s.n_pages = n_pages;
  p.s.max_pages = max_pages;
  p.s.page_shift = page_shift_of(page_size);
  p.s.capacity = max_pages * page_size;
  p.s.left = window_left;
  p.s.right = window_right;
  p.s.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634074);
  p.s.status = fa_host::status_word(dev);
  if (!p.s.status) return FA_ERR_LAUNCH;
  p.k = static_cast<const uint16_t*>(k_cache);
  p.k_page = strides[0];
  p.k_head = strides[1];
  p.k_token = strides[2];
  p.w = weights;
  p.w_page = strides[3];
  p.w_head = strides[4];
  p.decay = decay;
  p.group = H / Hk;
  if (T > 1) {  // 2^(31 + s) / T rounded up makes r / T too large by less than 2^-s <= 1 / T for r < 2^31
    int s = 0;
    while ((1ll << s) < T) ++s;
    p.t_mul = static_cast<unsigned>(((1ull << (31 + s)) + T - 1) / T);
    p.t_shift = s - 1;
  }
  const long long all_rows = static_cast<long long>(B) * H * T;
  return d == 64 ? launch_weights<64>(p, all_rows, page_size, sms, stream)
                 : launch_weights<128>(p, all_rows, page_size, sms, stream);
}

size_t fa_evict_workspace_bytes(int B, int Hk) {
  return B > 0 && Hk > 0 && static_cast<long long>(B) * Hk < (1ll << 28) ? EvictWorkspace(B, Hk).bytes : 0;
}

int fa_kv_evict(void* k_cache, void* v_cache, float* weights, const int* block_table, const int* table_out,
                int out_pages, const int* seq_lens, int* lens_out, int* shift, int* kept, const long long* strides,
                int B, int Hk, int d, int n_pages, int page_size, int max_pages, int budget, int recent, int sinks,
                int slack, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (!k_cache || !v_cache || !weights || !block_table || !seq_lens || !lens_out || !kept || !strides || !workspace)
    return FA_ERR_NULL;
  if (misaligned(k_cache, 16) || misaligned(v_cache, 16) || misaligned(workspace, 16)) return FA_ERR_ALIGN;
  const void* words[] = {weights, block_table, table_out, seq_lens, lens_out, shift, kept};
  for (const void* x : words)
    if (misaligned(x, 4)) return FA_ERR_ALIGN;
  if (d != 64 && d != 128) return FA_ERR_HEADDIM;
  if (B <= 0 || Hk <= 0 || static_cast<long long>(B) * Hk >= (1ll << 28) ||
      !page_sizes_ok(n_pages, page_size, max_pages))
    return FA_ERR_SHAPE;
  if (budget <= 0 || budget > kMaxKeys || recent < 0 || sinks < 0 || slack < 0 || slack > kMaxKeys - budget ||
      static_cast<long long>(recent) + sinks > budget)
    return FA_ERR_SHAPE;
  const int most = budget + slack;
  if (table_out && (out_pages <= 0 || static_cast<long long>(out_pages) * page_size > kMaxKeys ||
                    static_cast<long long>(out_pages) * page_size < most ||
                    (table_out == block_table && out_pages != max_pages)))
    return FA_ERR_SHAPE;
  for (int i = 0; i < 8; ++i)  // page, head and token strides of K, then V; page and head strides of the weights
    if (!stride_ok(strides[i], i < 6 ? 8 : 1)) return FA_ERR_STRIDE;
  int dev = -1, sms = 0;
  int st = fa_host::current_device(&dev, &sms);
  if (st != FA_OK) return st;
  const EvictWorkspace at(B, Hk);
  if (workspace_bytes < at.bytes) return FA_ERR_WORKSPACE;
  const void* ptrs[] = {k_cache, v_cache, weights, block_table, seq_lens, lens_out, kept, workspace};
  for (const void* x : ptrs)
    if (!fa_host::is_device_pointer(x, dev)) return FA_ERR_POINTER;
  if ((table_out && !fa_host::is_device_pointer(table_out, dev)) || (shift && !fa_host::is_device_pointer(shift, dev)))
    return FA_ERR_POINTER;
  fa::EvictParams p = {};
  void* const caches[2] = {k_cache, v_cache};
  for (int i = 0; i < 2; ++i) {
    p.cache[i] = static_cast<uint16_t*>(caches[i]);
    p.page[i] = strides[3 * i];
    p.head[i] = strides[3 * i + 1];
    p.token[i] = strides[3 * i + 2];
  }
  p.w = weights;
  p.w_page = strides[6];
  p.w_head = strides[7];
  p.w_vec = !misaligned(weights, 16) && strides[6] % 4 == 0 && strides[7] % 4 == 0;
  p.table = block_table;
  p.table_out = table_out ? table_out : block_table;
  p.lens = seq_lens;
  p.lens_out = lens_out;
  p.shift = shift;
  p.kept = kept;
  p.heads = static_cast<fa::EvictHead*>(workspace);
  p.B = B;
  p.Hk = Hk;
  p.n_pages = n_pages;
  p.max_pages = max_pages;
  p.out_pages = table_out ? out_pages : max_pages;
  p.page_shift = page_shift_of(page_size);
  p.capacity = max_pages * page_size;
  p.budget = budget;
  p.recent = recent;
  p.sinks = sinks;
  p.most = most;
  p.status = fa_host::status_word(dev);
  if (!p.status) return FA_ERR_LAUNCH;
  st = ready(dev);
  if (st != FA_OK) return st;
  const long long heads = static_cast<long long>(B) * Hk;
  st = launch_select(p, at, heads, stream);
  if (st != FA_OK) return st;
  return d == 64 ? launch_move<64>(p, heads, sms, stream) : launch_move<128>(p, heads, sms, stream);
}

}  // extern "C"
