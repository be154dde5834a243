// fa_rope.cu -- entry points of the rotary-position kernels: fa_rope and
// fa_kv_append.  See include/fa.h for their contracts.
#include <cmath>
#include <cstdint>

#include "fa.h"
#include "fa_host.h"
#include "fa_rope_kernel.cuh"

namespace {

// Three strides of one view: multiples of 8 elements (16-byte chunks), at
// least 0 (a broadcast input) or 1 (an output).
bool strides_ok(const long long* s, bool output) {
  for (int i = 0; i < 3; ++i)
    if (s[i] < (output ? 8 : 0) || (s[i] & 7) || s[i] >= (1ll << 40)) return false;
  return true;
}

fa::RopeView view(const long long* s) { return {s[0], s[1], s[2]}; }
fa::RopeView contiguous(int heads, int n, int d) {
  return {static_cast<long long>(heads) * n * d, static_cast<long long>(n) * d, d};
}

// Heads per CTA: the angles are computed once per token and CTA, so a CTA takes
// several heads; but enough CTAs are wanted that the last wave of them is short
// (3 x 4099 tokens, 32 heads: 33.5 us with 4 heads, 34.0 with 8, 41.2 with 16;
// 2 x 2000 of 40: 13.9, 13.2, 12.8, with 2 it takes 16.4).  Few
// tokens are spread over the SMs whatever the angles cost.
constexpr long long kCtasPerSm = 24;
constexpr long long kLeastHeads = 4;
constexpr long long kLeastCtasPerSm = 4;

template <int D, bool PAGED>
int launch(fa::RopeParams& p, int interleaved, int sms, cudaStream_t stream) {
  constexpr int kTokens = fa::kRopeThreads / (D / 16);
  const long long tiles = (p.tokens + kTokens - 1) / kTokens;
  const long long heads = static_cast<long long>(p.heads[0]) + p.heads[1] + (PAGED ? p.heads[2] : 0);
  long long groups = (kCtasPerSm * sms + tiles - 1) / tiles;
  if (groups > heads / kLeastHeads) groups = heads / kLeastHeads;
  const long long least = (kLeastCtasPerSm * sms + tiles - 1) / tiles;
  if (groups < least) groups = least;
  if (groups > heads) groups = heads;
  if (groups > 65535) groups = 65535;  // grid y
  p.heads_per_cta = static_cast<int>((heads + groups - 1) / groups);
  groups = (heads + p.heads_per_cta - 1) / p.heads_per_cta;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(groups));
  cfg.blockDim = dim3(fa::kRopeThreads);
  cfg.stream = stream;
  return fa_host::launched(interleaved ? cudaLaunchKernelEx(&cfg, fa::fa_rope_kernel<D, true, PAGED>, p)
                                       : cudaLaunchKernelEx(&cfg, fa::fa_rope_kernel<D, false, PAGED>, p));
}

bool misaligned(const void* p) { return reinterpret_cast<uintptr_t>(p) & 15u; }

}  // namespace

extern "C" {

int fa_rope(const void* q, const void* k, void* q_out, void* k_out, const double* inv_freq, const int* positions,
            long long position_stride, long long offset, const long long* strides, int B, int H, int Hk, int N, int d,
            int rot, float mag, int interleaved, int backward, cudaStream_t stream) {
  const bool has_k = Hk != 0;
  const bool noop = N == 0;
  if (!inv_freq || (!noop && (!q || !q_out || (has_k && (!k || !k_out))))) return FA_ERR_NULL;
  if (misaligned(q) || misaligned(q_out) || (has_k && (misaligned(k) || misaligned(k_out))) ||
      (reinterpret_cast<uintptr_t>(inv_freq) & 7u) || (reinterpret_cast<uintptr_t>(positions) & 3u))
    return FA_ERR_ALIGN;
  if (d != 64 && d != 128) return FA_ERR_HEADDIM;
  if (B <= 0 || H <= 0 || Hk < 0 || N < 0 || H > (1 << 20) || Hk > (1 << 20)) return FA_ERR_SHAPE;
  if (rot < 16 || rot > d || rot % 16 != 0) return FA_ERR_SHAPE;
  if ((interleaved & ~1) || (backward & ~1)) return FA_ERR_SHAPE;
  if (positions && position_stride != 0 && position_stride < N) return FA_ERR_SHAPE;
  if (!std::isfinite(mag)) return FA_ERR_SCALE;
  const long long tokens = static_cast<long long>(B) * N;
  if (tokens >= (1ll << 31)) return FA_ERR_SHAPE;
  if (strides && !(strides_ok(strides, false) && strides_ok(strides + 6, true) &&
                   (!has_k || (strides_ok(strides + 3, false) && strides_ok(strides + 9, true)))))
    return FA_ERR_STRIDE;
  if (noop) return FA_OK;
  int dev = -1, sms = 0;
  const int st = fa_host::current_device(&dev, &sms);
  if (st != FA_OK) return st;
  if (!fa_host::is_device_pointer(q, dev) || !fa_host::is_device_pointer(q_out, dev) ||
      (has_k && (!fa_host::is_device_pointer(k, dev) || !fa_host::is_device_pointer(k_out, dev))) ||
      !fa_host::is_device_pointer(inv_freq, dev) || (positions && !fa_host::is_device_pointer(positions, dev)))
    return FA_ERR_POINTER;
  fa::RopeParams p = {};
  p.src[0] = static_cast<const uint16_t*>(q);
  p.src[1] = static_cast<const uint16_t*>(k);
  p.dst[0] = static_cast<uint16_t*>(q_out);
  p.dst[1] = static_cast<uint16_t*>(k_out);
  if (strides) {
    for (int t = 0; t < 2; ++t) {
      p.src_s[t] = view(strides + 3 * t);
      p.dst_s[t] = view(strides + 6 + 3 * t);
    }
  } else {
    p.src_s[0] = p.dst_s[0] = contiguous(H, N, d);
    p.src_s[1] = p.dst_s[1] = contiguous(Hk, N, d);
  }
  p.heads[0] = H;
  p.heads[1] = Hk;
  p.inv_freq = inv_freq;
  p.positions = positions;
  p.pos_stride = position_stride;
  p.offset = offset;
  p.tokens = tokens;
  p.N = N;
  p.rot = rot;
  p.mag = mag;
  p.sin_sign = backward ? -1.f : 1.f;
  return d == 64 ? launch<64, false>(p, interleaved, sms, stream) : launch<128, false>(p, interleaved, sms, stream);
}

int fa_kv_append(const void* q, const void* k, const void* v, void* q_out, void* k_cache, void* v_cache,
                 const double* inv_freq, const int* block_table, const int* seq_lens, const int* new_lens,
                 const long long* strides, int B, int H, int Hk, int T, int d, int rot, int n_pages, int page_size,
                 int max_pages, long long offset, float mag, int interleaved, cudaStream_t stream) {
  const bool has_q = H != 0;
  const bool noop = T == 0;
  if (!strides || !block_table || !seq_lens || !k_cache || !v_cache || (rot != 0 && !inv_freq) ||
      (!noop && (!k || !v || (has_q && (!q || !q_out)))))
    return FA_ERR_NULL;
  if (misaligned(k) || misaligned(v) || misaligned(k_cache) || misaligned(v_cache) ||
      (has_q && (misaligned(q) || misaligned(q_out))) || (reinterpret_cast<uintptr_t>(inv_freq) & 7u) ||
      ((reinterpret_cast<uintptr_t>(block_table) | reinterpret_cast<uintptr_t>(seq_lens) |
        reinterpret_cast<uintptr_t>(new_lens)) & 3u))
    return FA_ERR_ALIGN;
  if (d != 64 && d != 128) return FA_ERR_HEADDIM;
  if (B <= 0 || H < 0 || Hk <= 0 || T < 0 || H > (1 << 20) || Hk > (1 << 20)) return FA_ERR_SHAPE;
  if (rot < 0 || rot > d || rot % 16 != 0 || (interleaved & ~1)) return FA_ERR_SHAPE;
  if (n_pages <= 0 || max_pages <= 0 || page_size < 16 || page_size > 256 || (page_size & (page_size - 1)))
    return FA_ERR_SHAPE;
  if (!std::isfinite(mag)) return FA_ERR_SCALE;
  const long long tokens = static_cast<long long>(B) * T;
  if (tokens >= (1ll << 31)) return FA_ERR_SHAPE;
  for (int t = 0; t < 6; ++t)  // q, k, v, q_out, k_cache, v_cache
    if (!((t == 0 || t == 3) && !has_q) && !strides_ok(strides + 3 * t, t >= 3)) return FA_ERR_STRIDE;
  if (noop) return FA_OK;
  int dev = -1, sms = 0;
  const int st = fa_host::current_device(&dev, &sms);
  if (st != FA_OK) return st;
  const void* ptrs[] = {k, v, k_cache, v_cache, block_table, seq_lens};
  for (const void* x : ptrs)
    if (!fa_host::is_device_pointer(x, dev)) return FA_ERR_POINTER;
  if ((has_q && (!fa_host::is_device_pointer(q, dev) || !fa_host::is_device_pointer(q_out, dev))) ||
      (rot != 0 && !fa_host::is_device_pointer(inv_freq, dev)) ||
      (new_lens && !fa_host::is_device_pointer(new_lens, dev)))
    return FA_ERR_POINTER;
  fa::RopeParams p = {};
  const void* src[3] = {q, k, v};
  void* dst[3] = {q_out, k_cache, v_cache};
  const int heads[3] = {H, Hk, Hk};
  for (int t = 0; t < 3; ++t) {
    p.src[t] = static_cast<const uint16_t*>(src[t]);
    p.dst[t] = static_cast<uint16_t*>(dst[t]);
    p.src_s[t] = view(strides + 3 * t);
    p.dst_s[t] = view(strides + 9 + 3 * t);
    p.heads[t] = heads[t];
  }
  p.inv_freq = inv_freq;
  p.offset = offset;
  p.tokens = tokens;
  p.N = T;
  p.rot = rot;
  p.mag = mag;
  p.sin_sign = 1.f;
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.new_lens = new_lens;
  p.n_pages = n_pages;
  p.max_pages = max_pages;
  while ((1 << p.page_shift) < page_size) ++p.page_shift;
  p.status = fa_host::status_word(dev);
  if (!p.status) return FA_ERR_LAUNCH;
  return d == 64 ? launch<64, true>(p, interleaved, sms, stream) : launch<128, true>(p, interleaved, sms, stream);
}

}  // extern "C"
