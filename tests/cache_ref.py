"""Plain 64-bit implementations of the cached keys' weights and of eviction (numpy,
sequence by sequence), and the tolerance the GPU tests derive for the weights.

A weight is decay W + sum_r p_r, p_r = exp(x_r), x_r = scale q_r . k - lse_r, with the
lse that the kernel was given.  e = 2^-24 is half an fp32 step relative to the value.
  The product q . k: d products added in fp32, at most d / 16 + 16 additions deep, each off by at
    most one step (the tensor cores cut bits off) of the sum of sizes: below 2^-18 a, a = scale
    sum_i |q_i k_i|, for d <= 128.
  The exponent: scale's rounding, lse times log2 e, the difference: 4 e (|scale q . k| + |lse|).
  ex2.approx: 2^-22 relative.
  So p is off by p (2^-18 a + 2^-22 (|scale q . k| + |lse| + 1)), and the sum of n of them and
  decay W by at most n + 8 more roundings of what is added:
      tol = sum p (2^-18 a + 2^-22 (|s| + |lse| + 1)) + (n + 8) 2^-24 (sum p + |decay W|).
"""
from __future__ import annotations

import numpy as np

from serving_ref import gather


def key_weights(q, lse, k_cache, weights, table, lens, new, left, right, scale, decay):
    """(weights afterwards, tolerance, which slots are written) for q [B, H, T, d], lse [B, H, T], caches
    [n_pages, Hk, page(, d)], all float64."""
    B, H, T, d = q.shape
    Hk, page = k_cache.shape[1:3]
    G = H // Hk
    out, tol = weights.copy(), np.zeros_like(weights)
    written = np.zeros(weights.shape, bool)
    for b in range(B):
        n, m = max(0, int(lens[b])), min(max(0, int(new[b])), T)
        if n == 0 or m == 0:
            continue
        j = np.arange(n)
        pos = n - m + np.arange(m)
        seen = np.ones((m, n), bool)
        if left >= 0:
            seen &= j >= pos[:, None] - left
        if right >= 0:
            seen &= j <= pos[:, None] + right
        pages = np.asarray(table[b])[j // page]
        for hk in range(Hk):
            k = gather(k_cache, table[b], n, hk)
            total, err = np.zeros(n), np.zeros(n)
            for h in range(hk * G, (hk + 1) * G):
                s = q[b, h, :m] @ k.T * scale
                a = np.abs(q[b, h, :m]) @ np.abs(k).T * scale
                rows = lse[b, h, :m, None]
                use = seen & ~np.isneginf(rows)
                with np.errstate(invalid="ignore", over="ignore"):
                    p = np.where(use, np.exp(np.where(use, s - rows, 0.0)), 0.0)
                    err += np.where(use & (p > 0), p * (2.0 ** -18 * a + 2.0 ** -22 * (np.abs(s) + np.abs(rows) + 1)), 0.0).sum(0)
                total += p.sum(0)
            old = np.where((j < n - m) & (decay != 0), decay * out[pages, hk, j % page], 0.0)
            out[pages, hk, j % page] = old + total
            tol[pages, hk, j % page] = err + (G * m + 8) * 2.0 ** -24 * (total + np.abs(old))
            written[pages, hk, j % page] = True
    return out, tol, written


def order(w):
    """A key that sorts as eviction ranks: NaN above everything, -0 as 0."""
    return np.where(np.isnan(w), np.inf, w + 0.0), np.isnan(w)


def kept_slots(w, n, budget, recent, sinks):
    """Slots of 0..n-1 that stay, by their weights w [n]."""
    free = np.arange(sinks, n - recent)
    value, nan = order(w[free])
    by_weight = free[np.lexsort((free, -value, ~nan))]  # NaN first, then the heaviest, then the lower slot
    stay = np.concatenate([np.arange(sinks), by_weight[:budget - sinks - recent], np.arange(n - recent, n)])
    return np.sort(stay)


def evict(arrays, weights, table, lens, budget, recent, sinks, slack, table_out=None):
    """(arrays afterwards, lengths, kept lists): arrays [n_pages, Hk, page(, d)] moved alike, the weights among them."""
    most = budget + slack
    B, (Hk, page) = len(lens), weights.shape[1:3]
    old = [a.copy() for a in arrays]
    new = [a.copy() for a in arrays]
    kept = np.full((B, Hk, most), -1, np.int32)
    out = np.zeros(B, np.int32)
    for b in range(B):
        n = max(0, int(lens[b]))
        out[b] = budget if n > most else n
        to = table[b] if table_out is None else table_out[b]
        for h in range(Hk):
            if n > most:
                stay = kept_slots(gather(weights[..., None], table[b], n, h)[:, 0], n, budget, recent, sinks)
            else:
                stay = np.arange(n)
            i = np.arange(len(stay))
            kept[b, h, i] = stay
            if len(stay):
                src, dst = np.asarray(table[b])[stay // page], np.asarray(to)[i // page]
                for a, o in zip(new, old):
                    a[dst, h, i % page] = o[src, h, stay % page]
    return new, out, kept
