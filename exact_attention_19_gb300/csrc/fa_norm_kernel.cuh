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
// Bound: memory, 6 bytes per element (x and dy read, dx written, bf16); then, with
// 16 warps to an SM, the way from a head's loads through its two sums to its
// stores.  Threads hold the elements that fa_rope_kernel's do (16 of a head, so its
// sums are D / 16 lanes', both in one pass), two heads' loads in flight, their angles
// in shared memory, and a CTA walks over an equal share of the line of (token tile, head)
// of q or of k with the 16 weight gradients of its elements in registers: they leave
// once, D sums per CTA, which a second kernel adds in the order of the CTAs (no
// atomics: results repeat bit for bit on one GPU).  Measured with the second kernel:
// 3 x 4099 tokens of 16 + 16 heads at d = 128, half turned, 59.9 us (5.0 TB/s), 8 x 1024
// of 12 + 12 at d = 64, 22.8 us.  Slower: angles in registers (61.7 and 23.2), three CTAs
// to an SM (with four heads in flight 59.8 and 24.5) or five (72 and 26.9; 80 and 29 with
// angles in registers, which spill), one head in flight (67 and 24.6), whole items of 8
// heads strided over the CTAs (66 and 24.4), x and dy through shared memory by
// asynchronous copies two to four heads ahead (82 and 20.6).
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

// Loaded again for each head, so that they hold no registers between.
__device__ __forceinline__ void own_angles(const float4* at, float* v) {
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
               : "r"(static_cast<unsigned>(__cvta_generic_to_shared(at)))
               : "memory");
}

template <int D, bool INTERLEAVED, int NORM>
__global__ void __launch_bounds__(kNormBwdThreads, kNormBwdCtasPerSm) fa_norm_bwd_kernel(const NormBwdParams p) {
  constexpr int kUnits = D / 16;  // threads per token
  constexpr int kTokens = kNormBwdThreads / kUnits;
  constexpr int kU = 2;  // heads in flight, four loads of 16 bytes each
  __shared__ unsigned long long freq[D / 2];
  __shared__ float sums[kNormBwdThreads / 32][D];
  __shared__ float4 angles[4][kNormBwdThreads];  // each thread's 8 cosines and sines
  __shared__ float4 weights[4][kUnits];  // elements 4 q .. of the 16 that each unit of a token holds
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the sum over CTAs waits for this grid's end
  const int t = static_cast<int>(blockIdx.x) < p.ctas[0] ? 0 : 1;
  bool broken = false;
  if (threadIdx.x < p.rot / 2) {
    const double w = __ldg(p.inv_freq + threadIdx.x);
    freq[threadIdx.x] = turns_per_position(w);
    broken = !finite(w);
  }
  const int u = threadIdx.x % kUnits;
  const bool turns = u < p.rot / 16;
  const int c0 = (turns && !INTERLEAVED) ? 8 * u : 16 * u;
  const int c1 = (turns && !INTERLEAVED) ? p.rot / 2 + 8 * u : 16 * u + 8;
  if (threadIdx.x < kUnits) {
    float w[16];
    load_weight16(p.weight[t], p.weight_f32, c0, c1, w);
#pragma unroll
    for (int q = 0; q < 4; ++q) weights[q][u] = make_float4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
  }
  broken = __syncthreads_or(broken) != 0;  // some frequency is NaN or infinite: its pairs become NaN
  float dw[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) dw[i] = 0.f;

  // this CTA's share of the line of (token tile, head): an equal one, of whole heads
  const int heads = p.heads[t], cta = static_cast<int>(blockIdx.x) - (t ? p.ctas[0] : 0);
  const long long line = (p.tokens + kTokens - 1) / kTokens * heads;
  const long long end = line * (cta + 1) / p.ctas[t];
  for (long long at = line * cta / p.ctas[t]; at < end;) {
    const long long tile = at / heads;
    const int h_lo = static_cast<int>(at - tile * heads);
    const int h_hi = static_cast<int>(min(static_cast<long long>(heads), h_lo + end - at));
    at += h_hi - h_lo;
    const long long tok = tile * kTokens + threadIdx.x / kUnits;
    if (tok >= p.tokens) continue;
    const int b = static_cast<int>(tok / p.N), n = static_cast<int>(tok - static_cast<long long>(b) * p.N);
    if (turns) {
      float c[8], s[8];
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
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        angles[q][threadIdx.x] = make_float4(c[4 * q], c[4 * q + 1], c[4 * q + 2], c[4 * q + 3]);
        angles[2 + q][threadIdx.x] = make_float4(s[4 * q], s[4 * q + 1], s[4 * q + 2], s[4 * q + 3]);
      }
    }
    const uint16_t* dy = p.dy[t] + b * p.dy_s[t].b + n * p.dy_s[t].n + h_lo * p.dy_s[t].h;
    const uint16_t* x = p.x[t] + b * p.x_s[t].b + n * p.x_s[t].n + h_lo * p.x_s[t].h;
    uint16_t* dx = p.dx[t] + b * p.dx_s[t].b + n * p.dx_s[t].n + h_lo * p.dx_s[t].h;
    for (int h = h_lo; h < h_hi; h += kU) {
      uint4 ga[kU], ge[kU], xa[kU], xe[kU];
#pragma unroll
      for (int i = 0; i < kU; ++i)
        if (h + i < h_hi) {
          ga[i] = *reinterpret_cast<const uint4*>(dy + c0);
          ge[i] = *reinterpret_cast<const uint4*>(dy + c1);
          xa[i] = *reinterpret_cast<const uint4*>(x + c0);
          xe[i] = *reinterpret_cast<const uint4*>(x + c1);
          dy += p.dy_s[t].h;
          x += p.x_s[t].h;
        }
#pragma unroll
      for (int i = 0; i < kU; ++i)
        if (h + i < h_hi) {
          float g[16], v[16];
          unpack16(ga[i], ge[i], g);
          unpack16(xa[i], xe[i], v);
          if (turns) {
            float c[8], s[8];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              own_angles(&angles[q][threadIdx.x], c + 4 * q);
              own_angles(&angles[2 + q][threadIdx.x], s + 4 * q);
            }
            rotate16<INTERLEAVED>(g, c, s);
          }
          // both sums over the head at once: of x^2, and of g w x, which r makes that of g w n
          float ss0, ss1, dot0, dot1, scale = 1.f;
          auto sums = [&]() {
            ss0 = ss1 = dot0 = dot1 = 0.f;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float4 w = weights[q][u];
              const int j = 4 * q;
              ss0 = fmaf(v[j], v[j], ss0);
              ss1 = fmaf(v[j + 1], v[j + 1], ss1);
              ss0 = fmaf(v[j + 2], v[j + 2], ss0);
              ss1 = fmaf(v[j + 3], v[j + 3], ss1);
              dot0 = fmaf(g[j] * w.x, v[j], dot0);
              dot1 = fmaf(g[j + 1] * w.y, v[j + 1], dot1);
              dot0 = fmaf(g[j + 2] * w.z, v[j + 2], dot0);
              dot1 = fmaf(g[j + 3] * w.w, v[j + 3], dot1);
            }
          };
          sums();
          float m = fmaf(head_sum<kUnits>(ss0 + ss1), 1.f / D, p.eps);
          if constexpr (NORM == kNormAnySize)
            if (!plain_mean(m)) {  // n and dw do not see the scale, dx takes it at the end
              scale = head_scale(m);
#pragma unroll
              for (int j = 0; j < 16; ++j) v[j] *= scale;
              sums();
              m = fmaf(head_sum<kUnits>(ss0 + ss1), 1.f / D, p.eps * scale * scale);
            }
          const float r = rsqrtf(m);
          const float mean = head_sum<kUnits>(dot0 + dot1) * r * (1.f / D);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float4 w = weights[q][u];
            const float w4[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int j = 4 * q + e;
              const float n = v[j] * r;
              dw[j] = fmaf(g[j], n, dw[j]);
              g[j] = r * fmaf(-mean, n, g[j] * w4[e]);
            }
          }
          if constexpr (NORM == kNormAnySize) {
#pragma unroll
            for (int j = 0; j < 16; ++j) g[j] *= scale;
          }
          pack16(g, ga[i], ge[i]);
          *reinterpret_cast<uint4*>(dx + c0) = ga[i];
          *reinterpret_cast<uint4*>(dx + c1) = ge[i];
          dx += p.dx_s[t].h;
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

// dweight = the sum of the CTAs' parts.  grid: 8 columns (a sector of each part) of q's, then of k's, to a CTA; thread
// 8 i + c adds column c of every 128th part from i on, then the 128 sums are added in pairs.
constexpr int kNormSumThreads = 1024;
template <int D>
__global__ void __launch_bounds__(kNormSumThreads) fa_norm_bwd_sum_kernel(const NormBwdParams p) {
  constexpr int kEach = kNormSumThreads / 8;
  __shared__ float sums[32][8];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int t = blockIdx.x / (D / 8), col = threadIdx.x % 8, i0 = threadIdx.x / 8;
  if (!p.dweight[t]) return;
  const int e = blockIdx.x % (D / 8) * 8 + col;
  const float* const part = p.part + static_cast<long long>(t ? p.ctas[0] : 0) * D + e;
  float v = 0.f;
#pragma unroll 8
  for (int i = i0; i < p.ctas[t]; i += kEach) v += part[static_cast<long long>(i) * D];
  v += __shfl_xor_sync(0xffffffffu, v, 8);
  v += __shfl_xor_sync(0xffffffffu, v, 16);
  if ((threadIdx.x & 31) < 8) sums[threadIdx.x / 32][col] = v;
  __syncthreads();
  if (threadIdx.x < 8) {
    v = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += sums[i][threadIdx.x];
    p.dweight[t][e] = v;
  }
}

}  // namespace fa
