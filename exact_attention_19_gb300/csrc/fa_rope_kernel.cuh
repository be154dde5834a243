// fa_rope_kernel.cuh -- rotary positions over [B, H, N, d] tensors, and the
// same rotation on the way into a paged K/V cache.
//
// Pair i of a head's rotated part at position p turns by the angle p * w_i:
//   y0 = mag (x0 cos - x1 sin),  y1 = mag (x1 cos + x0 sin)
// with (x0, x1) = (x[i], x[i + rot/2]) (half layout) or (x[2i], x[2i + 1])
// (interleaved).  The backward is the transpose: sin negated, same mag.
//
// The angle: w_i comes in 64 bits.  A CTA turns each once into a fixed-point
// number of turns per position modulo 1 (64 fraction bits: the double's 53-bit
// significand times 2^66 / 2 pi, shifted by its exponent and rounded), so that
// p * w_i modulo one turn is ONE wrapping 64-bit integer multiplication: an fp32
// product loses the angle from about p = 10^5 on, and fp64 arithmetic runs at a
// small fraction of the fp32 rate here.  The product is exact, its factor off by
// at most 2^-65 (rounding) + |w_i| 2^-72 (the constant's 64 bits) of a turn, so
// the angle is off by at most |p| (2^-65 + |w_i| 2^-72) turns: below 2^-33 for
// 32-bit positions and |w_i| <= 32, about 5e-5 rad at |p| = 2^48.
//
// Bound: memory, 4 bytes per element (bf16 read + write).  One thread owns 16
// elements (two 16-byte chunks, 8 pairs) of one token and walks over heads with
// its 8 cosines and sines in registers, so the angles are computed once per
// token and chunk, not per head.
// 4 x 8192 tokens, 32 + 8 heads of 128 (671 MB): 102.4 us, 6.6 TB/s, 97% of the
// copy rate; 3 x 4099 tokens, 16 + 16 heads (201 MB), 33.3 us, 89% (one and a
// half waves of CTAs); a call of 256 tokens 2.9 us, its launch.  Appending 4 x up
// to 2048 tokens, 32 + 2 x 8 heads (115 MB): 22.0 us, 77% (the page's index comes
// before the first store).
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace fa {

constexpr unsigned kStatusPage = 2u;  // FA_STATUS_PAGE

// Strides in elements of a [B, heads, N, d] view whose d is contiguous.
struct RopeView {
  long long b, h, n;
};

struct RopeParams {
  const uint16_t* src[3];  // q, k, v (v: append only, copied)
  uint16_t* dst[3];        // q, k outputs; append: q output, K cache, V cache
  RopeView src_s[3];
  RopeView dst_s[3];       // append: the caches' page, head and token strides
  int heads[3];            // heads of each tensor (0: absent)
  const double* inv_freq;  // [rot / 2], radians per position
  const int* positions;    // [B or 1, N] or nullptr (position = offset + token)
  long long pos_stride;    // N, or 0 for one row shared by the batch
  long long offset;
  long long tokens;        // B * N
  int N;
  int rot;
  int heads_per_cta;       // heads (counted over all tensors) one CTA walks over
  float mag, sin_sign;
  // append only
  const int* block_table;  // [B, max_pages]
  const int* seq_lens;     // [B], with the new tokens
  const int* new_lens;     // [B] or nullptr (N each)
  int n_pages, max_pages, page_shift;
  unsigned int* status;
};

// radians per position -> turns per position modulo 1, 64 fraction bits
__device__ __forceinline__ unsigned long long turns_per_position(double w) {
  constexpr unsigned long long kInv2Pi66 = 0xA2F9836E4E44152Aull;  // 2^66 / (2 pi)
  const unsigned long long bits = static_cast<unsigned long long>(__double_as_longlong(w));
  const int expo = static_cast<int>((bits >> 52) & 0x7ffu);
  const unsigned long long frac = bits & 0xfffffffffffffull;
  if (expo == 0 || expo == 0x7ff) return 0ull;  // zero, subnormal (below 2^-64 turns); not finite: see finite()
  const unsigned long long m = frac | (1ull << 52);
  // |w| = m 2^(expo - 1075); turns 2^64 = (m * kInv2Pi66) >> (1077 - expo)
  const unsigned long long lo = m * kInv2Pi66, hi = __umul64hi(m, kInv2Pi66);
  const int s = 1077 - expo;
  // to the nearest (ties away from zero)
  unsigned long long f;
  if (s >= 128) f = 0ull;
  else if (s > 64) f = ((hi >> (s - 65)) + 1ull) >> 1;
  else if (s == 64) f = hi + (lo >> 63);
  else if (s > 0) f = ((hi << (64 - s)) | (lo >> s)) + ((lo >> (s - 1)) & 1ull);
  else f = s > -64 ? lo << (-s) : 0ull;
  return (bits >> 63) ? 0ull - f : f;
}

// integer tests: fp64 comparisons run at a small fraction of the rate here
__device__ __forceinline__ bool finite(double w) { return (__double2hiint(w) & 0x7ff00000) != 0x7ff00000; }

// Cosine and sine of a 64-bit fraction of a turn, each with fp32's relative
// accuracy: a slow pair's sine at a small position is all that one element of the
// pair gets of the other, so an error that is small beside 1 only would be lost
// on most pairs and be all of a few results (base 500000, 128 elements, position
// 1: a sine of 2.5e-6).  The nearest quarter turn is taken off in integers; what is
// left, an eighth of a turn at most, is converted word by word (its size: the
// words of a small negative number would cancel) and goes into the Taylor sums up
// to a^9 and a^8, which for |a| <= pi / 4 leave 2^-28 and 2^-24.7 of the value.
__device__ __forceinline__ void cos_sin_turns(unsigned long long phase, float& c, float& s) {
  const unsigned quarter = static_cast<unsigned>((phase + (1ull << 61)) >> 62);
  const long long rest = static_cast<long long>(phase - (static_cast<unsigned long long>(quarter) << 62));
  const unsigned long long size = static_cast<unsigned long long>(rest < 0 ? -rest : rest);
  const float top = static_cast<float>(static_cast<unsigned>(size >> 32));
  const float m = fmaf(top, 4294967296.f, static_cast<float>(static_cast<unsigned>(size))) * 3.40612158e-19f;
  const float a = rest < 0 ? -m : m;  // size 2 pi 2^-64, signed
  const float z = a * a;
  float sn = fmaf(z, 2.75573192e-6f, -1.98412698e-4f);  // 1/9!, 1/7!, 1/5!, 1/3!
  sn = fmaf(z, sn, 8.33333333e-3f);
  sn = fmaf(z, sn, -1.66666667e-1f);
  sn = fmaf(a * z, sn, a);
  float cs = fmaf(z, 2.48015873e-5f, -1.38888889e-3f);  // 1/8!, 1/6!, 1/4!, 1/2!
  cs = fmaf(z, cs, 4.16666667e-2f);
  cs = fmaf(z, cs, -0.5f);
  cs = fmaf(z, cs, 1.0f);
  const float even = (quarter & 1u) ? sn : cs, odd = (quarter & 1u) ? cs : sn;
  c = ((quarter + 1u) & 2u) ? -even : even;
  s = (quarter & 2u) ? -odd : odd;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
// round to nearest even; `lo` in bits 0-15
__device__ __forceinline__ uint32_t rope_pack(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// The 16 elements (a: first chunk, b: second) of one head, rotated.
template <bool INTERLEAVED>
__device__ __forceinline__ void rotate16(uint4& a, uint4& b, const float (&c)[8], const float (&s)[8]) {
  uint32_t* const pa = &a.x;
  uint32_t* const pb = &b.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (INTERLEAVED) {
      const float a0 = bf16_lo(pa[i]), a1 = bf16_hi(pa[i]), b0 = bf16_lo(pb[i]), b1 = bf16_hi(pb[i]);
      pa[i] = rope_pack(fmaf(a0, c[i], -(a1 * s[i])), fmaf(a1, c[i], a0 * s[i]));
      pb[i] = rope_pack(fmaf(b0, c[4 + i], -(b1 * s[4 + i])), fmaf(b1, c[4 + i], b0 * s[4 + i]));
    } else {
      const float x0 = bf16_lo(pa[i]), x1 = bf16_hi(pa[i]), y0 = bf16_lo(pb[i]), y1 = bf16_hi(pb[i]);
      pa[i] = rope_pack(fmaf(x0, c[2 * i], -(y0 * s[2 * i])), fmaf(x1, c[2 * i + 1], -(y1 * s[2 * i + 1])));
      pb[i] = rope_pack(fmaf(y0, c[2 * i], x0 * s[2 * i]), fmaf(y1, c[2 * i + 1], x1 * s[2 * i + 1]));
    }
  }
}

constexpr int kRopeThreads = 128;

// grid: x = tiles of kRopeThreads / (D / 16) tokens, y = groups of heads.
// PAGED: k and v go to the cache slots of their sequence's pages, q to dst[0];
// a token past its sequence's new tokens, or whose slot lies outside the
// cache, is not written.
template <int D, bool INTERLEAVED, bool PAGED>
__global__ void __launch_bounds__(kRopeThreads) fa_rope_kernel(const RopeParams p) {
  constexpr int kUnits = D / 16;  // threads per token
  // head range of this CTA over q, then k, then v
  const int h_lo = blockIdx.y * p.heads_per_cta, h_hi = h_lo + p.heads_per_cta;
  // The frequencies as turns per position, once for the CTA's tokens (converted by every thread for its own
  // eight pairs, a call of 256 tokens took 3.9 us for 2.8, 2 x 2000 tokens of 32 + 8 heads 17.3 for 13.5).
  __shared__ unsigned long long freq[D / 2];
  static_assert(D / 2 <= kRopeThreads, "a thread converts one frequency");
  const bool angles = h_lo < p.heads[0] + p.heads[1];
  bool broken = false;
  if (angles && threadIdx.x < p.rot / 2) {
    const double w = __ldg(p.inv_freq + threadIdx.x);
    freq[threadIdx.x] = turns_per_position(w);
    broken = !finite(w);
  }
  broken = __syncthreads_or(broken) != 0;  // some frequency is NaN or infinite: its pairs become NaN
  const long long tok = static_cast<long long>(blockIdx.x) * (kRopeThreads / kUnits) + threadIdx.x / kUnits;
  const int u = threadIdx.x % kUnits;
  if (tok >= p.tokens) return;
  const int b = static_cast<int>(tok / p.N), n = static_cast<int>(tok - static_cast<long long>(b) * p.N);

  unsigned long long pos;  // modulo 2^64, as the phase is
  long long page = -1, slot = 0;  // the token's place in the cache; page: checked where it is used, so that the
                                  // first heads' loads need not wait for it
  if constexpr (PAGED) {
    const int len = p.seq_lens[b], fresh = p.new_lens ? min(p.new_lens[b], p.N) : p.N;
    const long long own = static_cast<long long>(len) - fresh + n;
    if (n >= fresh || own < 0) return;  // padding, or a padded entry of the batch
    pos = static_cast<unsigned long long>(p.offset) + own;
    if (h_hi > p.heads[0]) {
      const long long pi = own >> p.page_shift;
      if (pi < p.max_pages) page = p.block_table[static_cast<long long>(b) * p.max_pages + pi];
      slot = own & ((1ll << p.page_shift) - 1);
    }
  } else {
    pos = static_cast<unsigned long long>(p.offset) + (p.positions ? p.positions[b * p.pos_stride + n] : n);
  }

  // chunks of this thread: 8 rotation pairs, or 16 elements that pass through
  const bool turns = u < p.rot / 16;
  const int c0 = (turns && !INTERLEAVED) ? 8 * u : 16 * u;
  const int c1 = (turns && !INTERLEAVED) ? p.rot / 2 + 8 * u : 16 * u + 8;
  float c[8], s[8];
  if (turns && angles) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float sn, cs;
      cos_sin_turns(pos * freq[8 * u + i], cs, sn);
      if (broken && !finite(__ldg(p.inv_freq + 8 * u + i))) cs = sn = __int_as_float(0x7fffffff);
      c[i] = cs * p.mag;
      s[i] = sn * (p.mag * p.sin_sign);
    }
  }

  int first = 0;  // heads before this tensor
#pragma unroll
  for (int t = 0; t < (PAGED ? 3 : 2); ++t) {
    const int lo = max(h_lo - first, 0), hi = min(h_hi - first, p.heads[t]);
    first += p.heads[t];
    if (lo >= hi) continue;
    const uint16_t* const src = p.src[t] + b * p.src_s[t].b + n * p.src_s[t].n;
    // heads in flight, two loads of 16 bytes each (4 x 2048 appended: 22.0 us with 2, 24.1 with 4; 4 x 8192
    // rotated: 103.6 with 2, 102.5 with 4)
    constexpr int kU = PAGED ? 2 : 4;
    for (int h = lo; h < hi; h += kU) {
      uint4 a[kU], e[kU];
#pragma unroll
      for (int i = 0; i < kU; ++i)
        if (h + i < hi) {
          a[i] = *reinterpret_cast<const uint4*>(src + (h + i) * p.src_s[t].h + c0);
          e[i] = *reinterpret_cast<const uint4*>(src + (h + i) * p.src_s[t].h + c1);
        }
      uint16_t* dst = p.dst[t];
      if (PAGED && t > 0) {
        if (page < 0 || page >= p.n_pages) {  // the token has no slot
          if (u == 0) atomicOr(p.status, kStatusPage);
          break;
        }
        dst += page * p.dst_s[t].b + slot * p.dst_s[t].n;
      } else {
        dst += b * p.dst_s[t].b + n * p.dst_s[t].n;
      }
#pragma unroll
      for (int i = 0; i < kU; ++i)
        if (h + i < hi) {
          if (t < 2 && turns) rotate16<INTERLEAVED>(a[i], e[i], c, s);
          *reinterpret_cast<uint4*>(dst + (h + i) * p.dst_s[t].h + c0) = a[i];
          *reinterpret_cast<uint4*>(dst + (h + i) * p.dst_s[t].h + c1) = e[i];
        }
    }
  }
}

}  // namespace fa
