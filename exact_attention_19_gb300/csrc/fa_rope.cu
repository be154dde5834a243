// fa_rope.cu -- entry points of the rotary-position kernels: fa_rope and
// fa_kv_append, fa_norm_rope, fa_kv_append_norm and fa_norm_rope_bwd.  See
// include/fa.h for their contracts.
#include <cmath>
#include <cstdint>

#include "fa.h"
#include "fa_host.h"
#include "fa_norm_kernel.cuh"
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
// tokens are spread over the SMs whatever the angles cost.  The append with the norm, whose
// CTAs have more to begin with (the weights too) and more heads in flight, takes as many
// heads as leave the least number of CTAs: with that / with kCtasPerSm, 32 + 2 x 8 heads of
// 128, 4 x 2048 tokens 36.8 / 40.0 us, of 1 .. 2048 19.5 / 23.0, 2 x 8192 67.8 / 68.4, 32768
// 130 / 127; 12 + 2 x 12 of 64, 4 x 2048 11.9 / 15.1.
constexpr long long kCtasPerSm = 24;
constexpr long long kLeastHeads = 4;
constexpr long long kLeastCtasPerSm = 4;

template <int D, bool PAGED, int NORM>
int launch(fa::RopeParams& p, int interleaved, int sms, cudaStream_t stream) {
  constexpr int kTokens = fa::kRopeThreads / (D / 16);
  const long long tiles = (p.tokens + kTokens - 1) / kTokens;
  const long long heads = static_cast<long long>(p.heads[0]) + p.heads[1] + (PAGED ? p.heads[2] : 0);
  long long groups = NORM && PAGED ? 0 : (kCtasPerSm * sms + tiles - 1) / tiles;
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
  return fa_host::launched(interleaved ? cudaLaunchKernelEx(&cfg, fa::fa_rope_kernel<D, true, PAGED, NORM>, p)
                                       : cudaLaunchKernelEx(&cfg, fa::fa_rope_kernel<D, false, PAGED, NORM>, p));
}
template <bool PAGED, int NORM>
int launch(fa::RopeParams& p, int d, int interleaved, int sms, cudaStream_t stream) {
  return d == 64 ? launch<64, PAGED, NORM>(p, interleaved, sms, stream)
                 : launch<128, PAGED, NORM>(p, interleaved, sms, stream);
}
template <bool PAGED>
int launch(fa::RopeParams& p, int d, bool norm, int interleaved, int sms, cudaStream_t stream) {
  if (!norm) return launch<PAGED, fa::kNoNorm>(p, d, interleaved, sms, stream);
  return p.eps < fa::kNormLeastEps ? launch<PAGED, fa::kNormAnySize>(p, d, interleaved, sms, stream)
                                   : launch<PAGED, fa::kNorm>(p, d, interleaved, sms, stream);
}

bool misaligned(const void* p) { return reinterpret_cast<uintptr_t>(p) & 15u; }

// The norm of the calls that have one.
struct Norm {
  const void *q_weight, *k_weight;  // [d] or NULL
  int weights_f32;
  float eps;
};
int check_norm(const Norm& n) {
  if (misaligned(n.q_weight) || misaligned(n.k_weight)) return FA_ERR_ALIGN;
  if (n.weights_f32 & ~1) return FA_ERR_SHAPE;
  return std::isfinite(n.eps) && n.eps >= 0.f ? FA_OK : FA_ERR_SCALE;
}
bool norm_on_device(const Norm& n, int dev) {
  return (!n.q_weight || fa_host::is_device_pointer(n.q_weight, dev)) &&
         (!n.k_weight || fa_host::is_device_pointer(n.k_weight, dev));
}
void set_norm(fa::RopeParams& p, const Norm& n) {
  p.weight[0] = n.q_weight;
  p.weight[1] = n.k_weight;
  p.weight_f32 = n.weights_f32;
  p.eps = n.eps;
}

int rope_impl(const void* q, const void* k, void* q_out, void* k_out, const double* inv_freq, const int* positions,
              long long position_stride, long long offset, const long long* strides, int B, int H, int Hk, int N, int d,
              int rot, float mag, int interleaved, int backward, const Norm* norm, cudaStream_t stream) {
  const bool has_k = Hk != 0;
  const bool noop = N == 0;
  if ((!inv_freq && !(norm && rot == 0)) || (!noop && (!q || !q_out || (has_k && (!k || !k_out))))) return FA_ERR_NULL;
  if (misaligned(q) || misaligned(q_out) || (has_k && (misaligned(k) || misaligned(k_out))) ||
      (reinterpret_cast<uintptr_t>(inv_freq) & 7u) || (reinterpret_cast<uintptr_t>(positions) & 3u))
    return FA_ERR_ALIGN;
  if (d != 64 && d != 128) return FA_ERR_HEADDIM;
  if (B <= 0 || H <= 0 || Hk < 0 || N < 0 || H > (1 << 20) || Hk > (1 << 20)) return FA_ERR_SHAPE;
  if (rot < (norm ? 0 : 16) || rot > d || rot % 16 != 0) return FA_ERR_SHAPE;
  if ((interleaved & ~1) || (backward & ~1)) return FA_ERR_SHAPE;
  if (positions && position_stride != 0 && position_stride < N) return FA_ERR_SHAPE;
  if (!std::isfinite(mag)) return FA_ERR_SCALE;
  if (const int st = norm ? check_norm(*norm) : FA_OK; st != FA_OK) return st;
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
      (inv_freq && !fa_host::is_device_pointer(inv_freq, dev)) ||
      (positions && !fa_host::is_device_pointer(positions, dev)) || (norm && !norm_on_device(*norm, dev)))
    return FA_ERR_POINTER;
  fa::RopeParams p = {};
  if (norm) set_norm(p, *norm);
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
  return launch<false>(p, d, norm != nullptr, interleaved, sms, stream);
}

int append_impl(const void* q, const void* k, const void* v, void* q_out, void* k_cache, void* v_cache,
                const double* inv_freq, const int* block_table, const int* seq_lens, const int* new_lens,
                const int* shift, const long long* strides, int B, int H, int Hk, int T, int d, int rot, int n_pages,
                int page_size, int max_pages, long long offset, float mag, int interleaved, const Norm* norm,
                cudaStream_t stream) {
  const bool has_q = H != 0;
  const bool noop = T == 0;
  if (!strides || !block_table || !seq_lens || !k_cache || !v_cache || (rot != 0 && !inv_freq) ||
      (!noop && (!k || !v || (has_q && (!q || !q_out)))))
    return FA_ERR_NULL;
  if (misaligned(k) || misaligned(v) || misaligned(k_cache) || misaligned(v_cache) ||
      (has_q && (misaligned(q) || misaligned(q_out))) || (reinterpret_cast<uintptr_t>(inv_freq) & 7u) ||
      ((reinterpret_cast<uintptr_t>(block_table) | reinterpret_cast<uintptr_t>(seq_lens) |
        reinterpret_cast<uintptr_t>(new_lens) | reinterpret_cast<uintptr_t>(shift)) & 3u))
    return FA_ERR_ALIGN;
  if (d != 64 && d != 128) return FA_ERR_HEADDIM;
  if (B <= 0 || H < 0 || Hk <= 0 || T < 0 || H > (1 << 20) || Hk > (1 << 20)) return FA_ERR_SHAPE;
  if (rot < 0 || rot > d || rot % 16 != 0 || (interleaved & ~1)) return FA_ERR_SHAPE;
  if (n_pages <= 0 || max_pages <= 0 || page_size < 16 || page_size > 256 || (page_size & (page_size - 1)))
    return FA_ERR_SHAPE;
  if (!std::isfinite(mag)) return FA_ERR_SCALE;
  if (const int st = norm ? check_norm(*norm) : FA_OK; st != FA_OK) return st;
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
      (new_lens && !fa_host::is_device_pointer(new_lens, dev)) || (shift && !fa_host::is_device_pointer(shift, dev)) ||
      (norm && !norm_on_device(*norm, dev)))
    return FA_ERR_POINTER;
  fa::RopeParams p = {};
  if (norm) set_norm(p, *norm);
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
  p.shift = shift;
  p.n_pages = n_pages;
  p.max_pages = max_pages;
  while ((1 << p.page_shift) < page_size) ++p.page_shift;
  p.status = fa_host::status_word(dev);
  if (!p.status) return FA_ERR_LAUNCH;
  return launch<true>(p, d, norm != nullptr, interleaved, sms, stream);
}

// The CTAs of the norm's backward, and the sums they leave.
int bwd_ctas(int sms) { return fa::kNormBwdCtasPerSm * sms; }

template <int D, int NORM>
int launch_norm_bwd(fa::NormBwdParams& p, int interleaved, int sms, cudaStream_t stream) {
  constexpr int kTokens = fa::kNormBwdThreads / (D / 16);
  const long long tiles = (p.tokens + kTokens - 1) / kTokens;
  const long long grid = bwd_ctas(sms);
  // the line of (token tile, head) of each tensor is cut for its share of the CTAs
  const long long line[2] = {tiles * p.heads[0], tiles * p.heads[1]}, all = line[0] + line[1];
  long long ctas = all < grid ? all : grid;
  long long k = line[1] ? (ctas * line[1] + all - 1) / all : 0;  // k's CTAs, q's not none either
  if (k >= ctas) k = ctas - 1;
  if (all == 0) {  // no tokens: the weights' gradients are zeros
    k = p.heads[1] > 0;
    ctas = 1 + k;
  }
  p.ctas[0] = static_cast<int>(ctas - k);
  p.ctas[1] = static_cast<int>(k);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(fa::kNormBwdThreads);
  cfg.stream = stream;
  const int st = fa_host::launched(interleaved ? cudaLaunchKernelEx(&cfg, fa::fa_norm_bwd_kernel<D, true, NORM>, p)
                                               : cudaLaunchKernelEx(&cfg, fa::fa_norm_bwd_kernel<D, false, NORM>, p));
  if (st != FA_OK || (!p.dweight[0] && !p.dweight[1])) return st;
  return fa_host::launch_kernel(fa::fa_norm_bwd_sum_kernel<D>, 2 * (D / 8), fa::kNormSumThreads, 0, stream, p);
}

template <int D>
int launch_norm_bwd(fa::NormBwdParams& p, int interleaved, int sms, cudaStream_t stream) {
  return p.eps < fa::kNormLeastEps ? launch_norm_bwd<D, fa::kNormAnySize>(p, interleaved, sms, stream)
                                   : launch_norm_bwd<D, fa::kNorm>(p, interleaved, sms, stream);
}

}  // namespace

extern "C" {

int fa_rope(const void* q, const void* k, void* q_out, void* k_out, const double* inv_freq, const int* positions,
            long long position_stride, long long offset, const long long* strides, int B, int H, int Hk, int N, int d,
            int rot, float mag, int interleaved, int backward, cudaStream_t stream) {
  return rope_impl(q, k, q_out, k_out, inv_freq, positions, position_stride, offset, strides, B, H, Hk, N, d, rot, mag,
                   interleaved, backward, nullptr, stream);
}

int fa_norm_rope(const void* q, const void* k, void* q_out, void* k_out, const double* inv_freq, const void* q_weight,
                 const void* k_weight, const int* positions, long long position_stride, long long offset,
                 const long long* strides, int B, int H, int Hk, int N, int d, int rot, float mag, int interleaved,
                 float eps, int weights_f32, cudaStream_t stream) {
  const Norm norm = {q_weight, k_weight, weights_f32, eps};
  return rope_impl(q, k, q_out, k_out, inv_freq, positions, position_stride, offset, strides, B, H, Hk, N, d, rot, mag,
                   interleaved, 0, &norm, stream);
}

int fa_kv_append(const void* q, const void* k, const void* v, void* q_out, void* k_cache, void* v_cache,
                 const double* inv_freq, const int* block_table, const int* seq_lens, const int* new_lens,
                 const long long* strides, int B, int H, int Hk, int T, int d, int rot, int n_pages, int page_size,
                 int max_pages, long long offset, float mag, int interleaved, cudaStream_t stream) {
  return append_impl(q, k, v, q_out, k_cache, v_cache, inv_freq, block_table, seq_lens, new_lens, nullptr, strides, B, H,
                     Hk, T, d, rot, n_pages, page_size, max_pages, offset, mag, interleaved, nullptr, stream);
}

int fa_kv_append_norm(const void* q, const void* k, const void* v, void* q_out, void* k_cache, void* v_cache,
                      const double* inv_freq, const void* q_weight, const void* k_weight, const int* block_table,
                      const int* seq_lens, const int* new_lens, const int* shift, const long long* strides, int B,
                      int H, int Hk, int T, int d, int rot, int n_pages, int page_size, int max_pages,
                      long long offset, float mag, int interleaved, int norm, float eps, int weights_f32,
                      cudaStream_t stream) {
  if (norm & ~1) return FA_ERR_SHAPE;
  const Norm n = {q_weight, k_weight, weights_f32, eps};
  return append_impl(q, k, v, q_out, k_cache, v_cache, inv_freq, block_table, seq_lens, new_lens, shift, strides, B, H,
                     Hk, T, d, rot, n_pages, page_size, max_pages, offset, mag, interleaved, norm ? &n : nullptr,
                     stream);
}

size_t fa_norm_bwd_workspace_bytes(int d) {
  if (d != 64 && d != 128) return 0;
  int dev = -1, sms = 0;
  if (fa_host::current_device(&dev, &sms) != FA_OK) sms = 148;
  return static_cast<size_t>(bwd_ctas(sms)) * d * sizeof(float);
}

int fa_norm_rope_bwd(const void* dq, const void* dk, const void* q, const void* k, void* dq_out, void* dk_out,
                     float* dq_weight, float* dk_weight, const double* inv_freq, const void* q_weight,
                     const void* k_weight, const int* positions, long long position_stride, long long offset,
                     const long long* strides, int B, int H, int Hk, int N, int d, int rot, float mag,
                     int interleaved, float eps, int weights_f32, void* workspace, size_t workspace_bytes,
                     cudaStream_t stream) {
  const bool has_k = Hk != 0;
  const bool empty = N == 0;
  if ((!inv_freq && rot != 0) || (!empty && (!dq || !q || !dq_out || (has_k && (!dk || !k || !dk_out)))) ||
      ((dq_weight || dk_weight) && !workspace))
    return FA_ERR_NULL;
  const void* big[] = {dq, q, dq_out, dq_weight, dk_weight, workspace};
  for (const void* x : big)
    if (misaligned(x)) return FA_ERR_ALIGN;
  if ((has_k && (misaligned(dk) || misaligned(k) || misaligned(dk_out))) ||
      (reinterpret_cast<uintptr_t>(inv_freq) & 7u) || (reinterpret_cast<uintptr_t>(positions) & 3u))
    return FA_ERR_ALIGN;
  if (d != 64 && d != 128) return FA_ERR_HEADDIM;
  if (B <= 0 || H <= 0 || Hk < 0 || N < 0 || H > (1 << 20) || Hk > (1 << 20)) return FA_ERR_SHAPE;
  if (rot < 0 || rot > d || rot % 16 != 0 || (interleaved & ~1)) return FA_ERR_SHAPE;
  if (positions && position_stride != 0 && position_stride < N) return FA_ERR_SHAPE;
  if (!has_k && dk_weight) return FA_ERR_SHAPE;
  if (!std::isfinite(mag)) return FA_ERR_SCALE;
  const Norm norm = {q_weight, has_k ? k_weight : nullptr, weights_f32, eps};
  int st = check_norm(norm);
  if (st != FA_OK) return st;
  const long long tokens = static_cast<long long>(B) * N;
  if (tokens >= (1ll << 31)) return FA_ERR_SHAPE;
  if (strides)
    for (int t = 0; t < 6; ++t)  // dq, dk, q, k, dq_out, dk_out
      if ((has_k || t % 2 == 0) && !strides_ok(strides + 3 * t, t >= 4)) return FA_ERR_STRIDE;
  if (empty && !dq_weight && !dk_weight) return FA_OK;
  int dev = -1, sms = 0;
  st = fa_host::current_device(&dev, &sms);
  if (st != FA_OK) return st;
  if ((dq_weight || dk_weight) && workspace_bytes < fa_norm_bwd_workspace_bytes(d)) return FA_ERR_WORKSPACE;
  const void* need[] = {dq, q, dq_out};
  for (const void* x : need)
    if (!empty && !fa_host::is_device_pointer(x, dev)) return FA_ERR_POINTER;
  const void* maybe[] = {has_k ? dk : nullptr, has_k ? k : nullptr, has_k ? dk_out : nullptr, dq_weight, dk_weight,
                         rot ? inv_freq : nullptr, positions, dq_weight || dk_weight ? workspace : nullptr};
  for (const void* x : maybe)
    if (x && !fa_host::is_device_pointer(x, dev)) return FA_ERR_POINTER;
  if (!norm_on_device(norm, dev)) return FA_ERR_POINTER;
  fa::NormBwdParams p = {};
  const void* dy[2] = {dq, dk};
  const void* x[2] = {q, k};
  void* dx[2] = {dq_out, dk_out};
  for (int t = 0; t < 2; ++t) {
    p.dy[t] = static_cast<const uint16_t*>(dy[t]);
    p.x[t] = static_cast<const uint16_t*>(x[t]);
    p.dx[t] = static_cast<uint16_t*>(dx[t]);
    p.heads[t] = t ? Hk : H;
    const fa::RopeView all = contiguous(p.heads[t], N, d);
    p.dy_s[t] = strides ? view(strides + 3 * t) : all;
    p.x_s[t] = strides ? view(strides + 6 + 3 * t) : all;
    p.dx_s[t] = strides ? view(strides + 12 + 3 * t) : all;
  }
  p.inv_freq = inv_freq;
  p.positions = positions;
  p.pos_stride = position_stride;
  p.offset = offset;
  p.tokens = tokens;
  p.N = N;
  p.rot = rot;
  p.mag = mag;
  p.eps = eps;
  p.weight[0] = norm.q_weight;
  p.weight[1] = norm.k_weight;
  p.weight_f32 = weights_f32;
  p.part = static_cast<float*>(workspace);
  p.dweight[0] = dq_weight;
  p.dweight[1] = dk_weight;
  return d == 64 ? launch_norm_bwd<64>(p, interleaved, sms, stream) : launch_norm_bwd<128>(p, interleaved, sms, stream);
}

}  // extern "C"
