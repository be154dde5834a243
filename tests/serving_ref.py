"""Plain 64-bit implementations of the rotary and paged-cache operators (numpy,
sequence by sequence), and the tolerances the GPU tests derive from them.

Tolerances count roundings; u = 2^-8 is half a bf16 step relative to the value.

rope, kv_append: cos and sin carry a few fp32 roundings (2^-21 covers the angle's
  rounding to fp32, sincospi's error and the factor mag), the two products and
  their sum three more, the result one to bf16:
      |y - y_ref| <= u |y_ref| + 2^-20 |mag| (|x0| + |x1|).
O: every probability is rounded to bf16 before P V (u of it each), the result
  once more; scores, exponentials and sums are fp32 (below 2^-13 of each term
  for the sizes here):
      |O - O_ref| <= u |O_ref| + (u + 2^-12) sum_j p_j |v_j|.
LSE: fp32 scores: |LSE - ref| <= 2^-12 max(1, |ref|).
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -8


def rotate(x, positions, inv_freq, mag, interleaved, sign=1.0):
    """x [..., N, d] float64 turned by positions [N]; (result, |x0| + |x1| beside each element)."""
    half = len(inv_freq)
    r = 2 * half
    # angles in turns modulo one, exactly enough for any position: the product is split so that
    # nothing above one turn is lost
    pos = [int(p) for p in positions]
    from fractions import Fraction

    turns = np.array([[float((Fraction(p) * Fraction(float(w)) * INV_2PI) % 1) for w in inv_freq] for p in pos])
    a = 2.0 * np.pi * turns
    c, s = mag * np.cos(a), sign * mag * np.sin(a)
    first = slice(0, r, 2) if interleaved else slice(0, half)
    second = slice(1, r, 2) if interleaved else slice(half, r)
    y = x.copy()
    size = np.zeros_like(x)
    x0, x1 = x[..., first], x[..., second]
    y[..., first] = x0 * c - x1 * s
    y[..., second] = x1 * c + x0 * s
    size[..., first] = size[..., second] = abs(mag) * (np.abs(x0) + np.abs(x1))
    return y, size


def _inv_2pi():
    """1 / (2 pi) as a fraction, to 250 bits (Machin: pi = 16 atan(1/5) - 4 atan(1/239))."""
    from fractions import Fraction

    one = 1 << 300

    def atan_inv(n):
        total, term, k = 0, one // n, 0
        while term:
            total += (-1) ** k * (term // (2 * k + 1))
            term //= n * n
            k += 1
        return total

    pi = 4 * (4 * atan_inv(5) - atan_inv(239))
    return Fraction(one, 2 * pi)


INV_2PI = _inv_2pi()


def rope_tol(y_ref, size):
    return U * np.abs(y_ref) + 2.0 ** -20 * size


def attend(q, k, v, lo, hi, scale):
    """Rows q [n, d] over keys lo[i] <= j < hi[i] of k, v [L, d]: (O, LSE, sum_j p_j |v_j|)."""
    n, d = q.shape
    o, size, lse = np.zeros((n, d)), np.zeros((n, d)), np.full(n, -np.inf)
    for i in range(n):
        a, b = max(0, int(lo[i])), int(hi[i])
        if a >= b:
            continue
        s = (k[a:b] @ q[i]) * scale
        m = s.max()
        e = np.exp(s - m)
        lse[i] = m + np.log(e.sum())
        p = e / e.sum()
        o[i] = p @ v[a:b]
        size[i] = p @ np.abs(v[a:b])
    return o, lse, size


def gather(cache, pages, n, hk):
    """Keys 0..n-1 of one head: [n, d] from a cache [n_pages, Hk, page, d]."""
    page = cache.shape[2]
    j = np.arange(n)
    return cache[np.asarray(pages)[j // page] if n else np.zeros(0, int), hk, j % page]


def paged(q, k_cache, v_cache, table, lens, new, left, right, scale, prefix_pages=None, prefix_len=0):
    """fwd_paged / fwd_prefix in 64 bits: (O, LSE, size) shaped [B, H, T, ...]."""
    B, H, T, d = q.shape
    Hk = k_cache.shape[1]
    G = H // Hk
    o, size = np.zeros((B, H, T, d)), np.zeros((B, H, T, d))
    lse = np.full((B, H, T), -np.inf)
    for b in range(B):
        n, m = max(0, int(lens[b])), min(max(0, int(new[b])), T)
        for h in range(H):
            k, v = (gather(c, table[b], n, h // G) for c in (k_cache, v_cache))
            if prefix_len:
                k = np.concatenate([gather(k_cache, prefix_pages, prefix_len, h // G), k])
                v = np.concatenate([gather(v_cache, prefix_pages, prefix_len, h // G), v])
            pos = n - m + np.arange(m)  # own positions
            lo = np.zeros(m, int) if left < 0 else np.maximum(0, pos - left)
            hi = np.full(m, n) if right < 0 else np.minimum(n, pos + right + 1)
            if prefix_len:
                hi = np.where(pos >= 0, prefix_len + hi, 0)
            o[b, h, :m], lse[b, h, :m], size[b, h, :m] = attend(q[b, h, :m], k, v, lo, hi, scale)
    return o, lse, size


def check_attention(o, lse, ref, what=""):
    o_ref, lse_ref, size = ref
    empty = np.isneginf(lse_ref)
    assert np.array_equal(np.isneginf(lse), empty), f"{what}: rows without a key differ"
    assert np.all(np.isfinite(o)), f"{what}: non-finite O"
    over = np.abs(o - o_ref) - (U * np.abs(o_ref) + (U + 2.0 ** -12) * size)
    assert np.all(over <= 0), f"{what}: O off by up to {np.abs(o - o_ref).max():.3e}, over its bound by {over.max():.3e}"
    d = np.abs(np.where(empty, 0.0, lse) - np.where(empty, 0.0, lse_ref))
    tol = 2.0 ** -12 * np.maximum(1.0, np.abs(np.where(empty, 0.0, lse_ref)))
    assert np.all(d <= tol), f"{what}: LSE off by {d.max():.3e}"
