"""Plain 64-bit implementations of the norm with the rotation and of its gradients
(numpy), and the tolerances the GPU tests derive from them.

Roundings, with u = 2^-8 half a bf16 step and e = 2^-24 half an fp32 step, both
relative to the value.

1 / sqrt(mean x^2 + eps): 16 squares of a thread in two sums of 8 (8 roundings
  each), their sum, 3 lane sums, one product and addition: at most 13 e of a sum of
  positive terms, half of it after the root; rsqrtf's own 2^-22 (2 units in the last
  place): below 11 e.  With the two products of r, weight and x: 13 e < 2^-20.
y = R (n w): the rotation's 2^-20 (see serving_ref) on top, one rounding to bf16:
      |y - y_ref| <= u |y_ref| + 2^-19 s,   s = |mag| (|n0 w0| + |n1 w1|) of the pair.
dx = r (g w - n m), m = mean(g w n), g = R^T dy with error 2^-20 G, G = |mag| (|dy0| +
  |dy1|) of the pair: with U = G |w| >= |g w| and A = mean(U |n|), m is off by at most
  A (2^-20 from g, 2^-20 from n, 13 e from the sum) and every other step by 2^-20 at most:
      |dx - dx_ref| <= u |dx_ref| + 2^-18 r (U + |n| A).
dw = sum g n: each term off by 2^-19 G |n|, plus one rounding for every addition that a
  term goes through.  A thread adds its own terms one after another (at most 256 in the
  tests here), then 3 lanes, 4 warps and the CTAs (at most 64 and 32): below 512 e = 2^-15:
      |dw - dw_ref| <= (2^-19 + 2^-15) sum G |n|.
"""
from __future__ import annotations

import numpy as np

import serving_ref as ref

U = ref.U


def normed(x, eps):
    """(x / rms, 1 / rms) of each head of float64 x [..., d]."""
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return x * r, r


def _turn(x, positions, inv_freq, mag, interleaved, sign=1.0):
    """serving_ref.rotate, with its size beside every element (|x| beside those that do not turn)."""
    if inv_freq is None:
        return x, np.abs(x)
    y, size = ref.rotate(x, positions, inv_freq, mag, interleaved, sign)
    turned = np.zeros(x.shape[-1], bool)
    turned[:2 * len(inv_freq)] = True
    return y, np.where(turned, size, np.abs(x))


def norm_rope(x, weight, eps, positions, inv_freq, mag, interleaved):
    """x [..., N, d]: (y, bound)."""
    n, _ = normed(x, eps)
    y, size = _turn(n * weight, positions, inv_freq, mag, interleaved)
    return y, U * np.abs(y) + 2.0 ** -19 * size


def norm_rope_bwd(dy, x, weight, eps, positions, inv_freq, mag, interleaved):
    """dy, x [..., N, d]: (dx, bound, dw, bound)."""
    g, size = _turn(dy, positions, inv_freq, mag, interleaved, -1.0)
    n, r = normed(x, eps)
    u = g * weight
    dx = r * (u - n * (u * n).mean(-1, keepdims=True))
    big = size * np.abs(weight)
    bound = U * np.abs(dx) + 2.0 ** -18 * r * (big + np.abs(n) * (big * np.abs(n)).mean(-1, keepdims=True))
    axes = tuple(range(x.ndim - 1))
    return dx, bound, (g * n).sum(axes), (2.0 ** -19 + 2.0 ** -15) * (size * np.abs(n)).sum(axes)
