// fa_norm_kernel.cuh -- gradients of the norm of each head with the rotation
// (forward: fa_rope_kernel with NORM).
//
// Forward, for one head x of one token, R its rotation:
//   r = 1 / sqrt(mean x^2 + eps),  n = x r,  y = R (n w).
// Backward, from the gradient dy of y:
//   g = R^T dy,  dw = sum over tokens and heads of g n,
//   u = g w,  dx = r (u - n mean(u n)).
// r is found again from x (16 multiply-adds beside 96 bytes moved), so the
// forward leaves nothing behind.
//
// Bound: memory, 6 bytes per element (x and dy read, dx written, bf16).  Threads
// hold the elements that fa_rope_kernel's do (16 of a head, so the two sums of a
// head are D / 16 lanes'), and a CTA walks over (token tile, head group) items of
// q or of k with the 16 weight gradients of its elements in registers: they leave
// once, D sums per CTA, which a second kernel adds in the order of the CTAs (no
// atomics: results repeat bit for bit on one GPU).
#pragma once

#include "fa_rope_kernel.cuh"

namespace fa {

struct NormBwdParams {
  const uint16_t* dy[2];  // q, k
  const uint16_t* x[2];
  uint16_t* dx[2];
  RopeView dy_s[2], x_s[2], dx_s[2];
  int heads[2];            // heads of each (k's may be 0)
  int ctas[2];             // CTAs that walk over each
  int heads_per_item;
  const double* inv_freq;  // [rot / 2] (rot 0: not read)
  const int* positions;
  long long pos_stride, offset, tokens;
  int N, rot;
  float mag, eps;
  const void* weight[2];
  int weight_f32;
  float* part;        // [ctas[0] + ctas[1], D]
  float* dweight[2];  // [D] or nullptr
};

constexpr int kNormBwdThreads = 128;
constexpr int kNormBwdCtasPerSm = 4;

template <int D, bool INTERLEAVED>
__global__ void __launch_bounds__(kNormBwdThreads, kNormBwdCtasPerSm) fa_norm_bwd_kernel(const NormBwdParams p) {
  constexpr int kUnits = D / 16;  // threads per token
  constexpr int kTokens = kNormBwdThreads / kUnits;
  constexpr int kU = 2;  // heads in flight, four loads of 16 bytes each
  __shared__ unsigned long long freq[D / 2];
  __shared__ float sums[kNormBwdThreads / 32][D];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the sum over CTAs waits for this grid's end
  bool broken = false;
  if (threadIdx.x < p.rot / 2) {
    const double w = __ldg(p.inv_freq + threadIdx.x);
    freq[threadIdx.x] = turns_per_position(w);
    broken = !finite(w);
  }
  broken = __syncthreads_or(broken) != 0;  // some frequency is NaN or infinite: its pairs become NaN
  const int t = static_cast<int>(blockIdx.x) < p.ctas[0] ? 0 : 1;
  const int u = threadIdx.x % kUnits;
  const bool turns = u < p.rot / 16;
  const int c0 = (turns && !INTERLEAVED) ? 8 * u : 16 * u;
  const int c1 = (turns && !INTERLEAVED) ? p.rot / 2 + 8 * u : 16 * u + 8;
  float weight[16], dw[16];
  load_weight16(p.weight[t], p.weight_f32, c0, c1, weight);
#pragma unroll
  for (int i = 0; i < 16; ++i) dw[i] = 0.f;

  const int groups = (p.heads[t] + p.heads_per_item - 1) / p.heads_per_item;
  const long long items = (p.tokens + kTokens - 1) / kTokens * groups;
  for (long long item = blockIdx.x - (t ? p.ctas[0] : 0); item < items; item += p.ctas[t]) {
    const long long tile = item / groups;
    const long long tok = tile * kTokens + threadIdx.x / kUnits;
    if (tok >= p.tokens) continue;
    const int h_lo = static_cast<int>(item - tile * groups) * p.heads_per_item;
    const int h_hi = min(p.heads[t], h_lo + p.heads_per_item);
    const int b = static_cast<int>(tok / p.N), n = static_cast<int>(tok - static_cast<long long>(b) * p.N);
    float c[8], s[8];
    if (turns) {
      const unsigned long long pos =
          static_cast<unsigned long long>(p.offset) + (p.positions ? p.positions[b * p.pos_stride + n] : n);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float sn, cs;
        cos_sin_turns(pos * freq[8 * u + i], cs, sn);
        if (broken && !finite(__ldg(p.inv_freq + 8 * u + i))) cs = sn = __int_as_float(0x7fffffff);
        c[i] = cs * p.mag;
        s[i] = sn * -p.mag;
      }
    }
    const uint16_t* const dy = p.dy[t] + b * p.dy_s[t].b + n * p.dy_s[t].n;
    const uint16_t* const x = p.x[t] + b * p.x_s[t].b + n * p.x_s[t].n;
    uint16_t* const dx = p.dx[t] + b * p.dx_s[t].b + n * p.dx_s[t].n;
    for (int h = h_lo; h < h_hi; h += kU) {
      uint4 ga[kU], ge[kU], xa[kU], xe[kU];
#pragma unroll
      for (int i = 0; i < kU; ++i)
        if (h + i < h_hi) {
          ga[i] = *reinterpret_cast<const uint4*>(dy + (h + i) * p.dy_s[t].h + c0);
          ge[i] = *reinterpret_cast<const uint4*>(dy + (h + i) * p.dy_s[t].h + c1);
          xa[i] = *reinterpret_cast<const uint4*>(x + (h + i) * p.x_s[t].h + c0);
          xe[i] = *reinterpret_cast<const uint4*>(x + (h + i) * p.x_s[t].h + c1);
        }
#pragma unroll
      for (int i = 0; i < kU; ++i)
        if (h + i < h_hi) {
          float g[16], v[16];
          unpack16(ga[i], ge[i], g);
          unpack16(xa[i], xe[i], v);
          if (turns) rotate16<INTERLEAVED>(g, c, s);
          const float r = inverse_rms<D>(v, p.eps);
          float dot = 0.f;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            v[j] *= r;
            dw[j] = fmaf(g[j], v[j], dw[j]);
            g[j] *= weight[j];
            dot = fmaf(g[j], v[j], dot);
          }
          dot = head_sum<kUnits>(dot) * (1.f / D);
#pragma unroll
          for (int j = 0; j < 16; ++j) g[j] = r * fmaf(-dot, v[j], g[j]);
          pack16(g, ga[i], ge[i]);
          *reinterpret_cast<uint4*>(dx + (h + i) * p.dx_s[t].h + c0) = ga[i];
          *reinterpret_cast<uint4*>(dx + (h + i) * p.dx_s[t].h + c1) = ge[i];
        }
    }
  }

  if (!p.dweight[t]) return;
  // lanes u, u + kUnits, ... of a warp hold the same elements; then the warps
#pragma unroll
  for (int i = 0; i < 16; ++i)
#pragma unroll
    for (int o = kUnits; o < 32; o <<= 1) dw[i] += __shfl_xor_sync(0xffffffffu, dw[i], o);
  if ((threadIdx.x & 31) < kUnits) {
#pragma unroll
    for (int i = 0; i < 16; ++i) sums[threadIdx.x / 32][i < 8 ? c0 + i : c1 + i - 8] = dw[i];
  }
  __syncthreads();
  for (int e = threadIdx.x; e < D; e += kNormBwdThreads) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kNormBwdThreads / 32; ++w) v += sums[w][e];
    p.part[static_cast<long long>(blockIdx.x) * D + e] = v;
  }
}

// dweight = the sum of the CTAs' parts.  grid: 32 columns of q's, then of k's, to a CTA; a warp takes every 32nd part.
template <int D>
__global__ void __launch_bounds__(1024) fa_norm_bwd_sum_kernel(const NormBwdParams p) {
  __shared__ float sums[32][33];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int t = blockIdx.x / (D / 32), lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e = blockIdx.x % (D / 32) * 32 + lane;
  if (!p.dweight[t]) return;
  const float* const part = p.part + static_cast<long long>(t ? p.ctas[0] : 0) * D + e;
  float v = 0.f;
#pragma unroll 4
  for (int i = warp; i < p.ctas[t]; i += 32) v += part[static_cast<long long>(i) * D];
  sums[warp][lane] = v;
  __syncthreads();
  if (warp == 0) {
    v = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += sums[i][lane];
    p.dweight[t][e] = v;
  }
}

}  // namespace fa
