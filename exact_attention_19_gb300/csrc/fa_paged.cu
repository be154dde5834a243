// fa_paged.cu -- entry points of attention over the paged cache: fa_fwd_paged,
// fa_fwd_prefix and their workspace size.  See include/fa.h for their contracts.
#include <atomic>
#include <cmath>
#include <cstdint>

#include "fa.h"
#include "fa_host.h"
#include "fa_paged_kernel.cuh"

namespace {

constexpr int kMaxKeys = 1 << 30;  // tokens of a sequence or a prefix: tile arithmetic stays within an int

std::atomic<bool> g_ready[fa_host::kMaxDevices];

template <int D>
bool opt_in() {
  return cudaFuncSetAttribute(fa::fa_paged_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(fa::PagedCfg<D>::kSmemBytes)) == cudaSuccess;
}

// The kernels' shared-memory opt-in, once per device (a repeated call is harmless).
int ready(int dev) {
  if (g_ready[dev].load(std::memory_order_acquire)) return FA_OK;
  if (!opt_in<64>() || !opt_in<128>()) return FA_ERR_LAUNCH;
  g_ready[dev].store(true, std::memory_order_release);
  return FA_OK;
}

// 4-D map over a cache: (d, token of the page, K/V head, page), 128-byte
// swizzle, `rows` tokens x 64 elements per box.
bool make_cache_map(CUtensorMap* map, const void* ptr, int d, int page, int Hk, int n_pages, const long long* s,
                    int rows) {
  fa_host::EncodeTiledFn enc = fa_host::encode_fn();
  if (!enc) return false;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(page), static_cast<cuuint64_t>(Hk),
                        static_cast<cuuint64_t>(n_pages)};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(s[2]) * 2u, static_cast<cuuint64_t>(s[1]) * 2u,
                           static_cast<cuuint64_t>(s[0]) * 2u};
  cuuint32_t box[4] = {64u, static_cast<cuuint32_t>(rows), 1u, 1u};
  cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(ptr), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t up16(size_t n) { return (n + 15) / 16 * 16; }

// Parts of the workspace, in order; every size is a multiple of 16 bytes.
struct Layout {
  size_t plan, piece_o, piece_l, whole_o, whole_l;
  size_t bytes() const { return plan + piece_o + piece_l + whole_o + whole_l; }
};
Layout layout(int B, int H, int T, int d, bool prefix, int sms) {
  const size_t ctas = 2 * static_cast<size_t>(sms);
  const size_t rows = static_cast<size_t>(B) * H * T;
  Layout l;
  l.plan = up16((static_cast<size_t>(B) + 3) * sizeof(long long));
  l.piece_o = 2 * ctas * 16 * d * sizeof(float);
  l.piece_l = 2 * ctas * 16 * sizeof(float);
  l.whole_o = prefix ? 2 * rows * d * sizeof(float) : 0;
  l.whole_l = prefix ? up16(2 * rows * sizeof(float)) : 0;
  return l;
}

template <int D>
int launch(const CUtensorMap& mk, const CUtensorMap& mv, const fa::PagedParams& p, int ctas, long long rows,
           cudaStream_t stream) {
  using C = fa::PagedCfg<D>;
  fa::fa_paged_kernel<D><<<static_cast<unsigned>(ctas), C::kThreads, C::kSmemBytes, stream>>>(mk, mv, p);
  if (cudaGetLastError() != cudaSuccess) return FA_ERR_LAUNCH;
  // programmatic dependent launch: the merge's CTAs may be scheduled while the
  // last parts are computed and wait on the device for that grid's completion
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(rows));
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, fa::fa_paged_merge_kernel<D, C::kRows, C::kTile>, p);
  return (e == cudaSuccess && cudaGetLastError() == cudaSuccess) ? FA_OK : FA_ERR_LAUNCH;
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
  if (static_cast<long long>(max_pages) * page_size > kMaxKeys || rows >= (1ll << 31) ||
      static_cast<long long>(B) * H >= (1ll << 31))
    return FA_ERR_SHAPE;
  if (!std::isfinite(scale) || !(scale > 0.f)) return FA_ERR_SCALE;
  for (int i = 0; i < 6; ++i)  // page, head and token strides of K, then of V; a tensor map's limit is 2^40 bytes
    if (strides[i] < 8 || (strides[i] & 7) || strides[i] >= (1ll << 39)) return FA_ERR_STRIDE;
  if (noop) return FA_OK;
  int dev = -1, sms = 0;
  int st = fa_host::current_device(&dev, &sms);
  if (st != FA_OK) return st;
  const Layout l = layout(B, H, T, d, prefix_len > 0, sms);
  if (workspace_bytes < l.bytes()) return FA_ERR_WORKSPACE;
  const void* ptrs[] = {q, k_cache, v_cache, o, lse, workspace, block_table, seq_lens};
  for (const void* x : ptrs)
    if (!fa_host::is_device_pointer(x, dev)) return FA_ERR_POINTER;
  if ((new_lens && !fa_host::is_device_pointer(new_lens, dev)) ||
      (prefix_len > 0 && !fa_host::is_device_pointer(prefix_pages, dev)))
    return FA_ERR_POINTER;
  st = ready(dev);
  if (st != FA_OK) return st;
  CUtensorMap mk, mv;
  if (!make_cache_map(&mk, k_cache, d, page_size, Hk, n_pages, strides, 16) ||
      !make_cache_map(&mv, v_cache, d, page_size, Hk, n_pages, strides + 3, 16))
    return FA_ERR_LAUNCH;
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
  char* at = static_cast<char*>(workspace);
  p.plan = reinterpret_cast<long long*>(at);
  p.piece_o = reinterpret_cast<float*>(at += l.plan);
  p.piece_l = reinterpret_cast<float*>(at += l.piece_o);
  p.whole_o = reinterpret_cast<float*>(at += l.piece_l);
  p.whole_l = reinterpret_cast<float*>(at += l.whole_o);
  p.status = fa_host::status_word(dev);
  if (!p.status) return FA_ERR_LAUNCH;
  return d == 64 ? launch<64>(mk, mv, p, 2 * sms, rows, stream) : launch<128>(mk, mv, p, 2 * sms, rows, stream);
}

}  // namespace

extern "C" {

size_t fa_paged_workspace_bytes(int B, int H, int Hk, int T, int d, int prefix_len) {
  if (B <= 0 || H <= 0 || Hk <= 0 || H % Hk != 0 || T <= 0 || (d != 64 && d != 128) || prefix_len < 0) return 0;
  int dev = -1, sms = 0;
  if (fa_host::current_device(&dev, &sms) != FA_OK) sms = 148;
  return layout(B, H, T, d, prefix_len > 0, sms).bytes();
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
