"""kv_weights where a cluster has many units, of which whole runs are seen by no row, or by none of one CTA's: against
the definition in 64 bits, with cache_ref's tolerance, on the GPU (the sizes are large)."""
import math

import numpy as np
import pytest

import weights_roles as roles

torch = pytest.importorskip("torch")

from test_cache_gpu import Cache, bits, i32, rand  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import exact_attention_19_gb300 as mod
    from exact_attention_19_gb300 import build

    build.build()
    mod.load()
    return mod


@pytest.fixture(autouse=True)
def _status(fa):
    fa.fa_fwd_status(None, clear=True)
    yield
    torch.cuda.synchronize()
    st, word = fa.fa_fwd_status(None, clear=True)
    assert st == 0, f"status word {word:#x}"


def definition(q, lse, k, old, n, m, left, decay):
    """(weights, tolerance) of one sequence and K/V head: q [G, m, d], lse [G, m], k [n, d], old [n]."""
    q, k = q.double(), k.double()
    scale = 1.0 / math.sqrt(q.shape[-1])
    j0 = max(0, n - m - left) if left >= 0 else 0  # the keys before are seen by no row
    j, pos = torch.arange(j0, n, device=q.device), n - m + torch.arange(m, device=q.device)[:, None]
    seen = j <= pos
    if left >= 0:
        seen &= j >= pos - left
    total, err = torch.zeros(2, n, dtype=torch.float64, device=q.device)
    for g in range(q.shape[0]):
        s, a = q[g] @ k[j0:].T * scale, q[g].abs() @ k[j0:].abs().T * scale
        row = lse[g, :, None].double()
        p = torch.where(seen, (s - row).exp(), torch.zeros((), dtype=torch.float64, device=q.device))
        total[j0:] += p.sum(0)
        err[j0:] += (p * (2.0 ** -18 * a + 2.0 ** -22 * (s.abs() + row.abs() + 1))).sum(0)
    kept = torch.zeros_like(total)
    if decay:
        kept[:n - m] = decay * old[:n - m].double()
    return kept + total, err + (q.shape[0] * m + 8) * 2.0 ** -24 * (total + kept.abs())


def check(fa, c, B, H, Hk, T, lens, new, left, decay, table):
    """One call against the definition; `table` is the cache's, or wider."""
    fresh = [T] * B if new is None else new
    q, window = rand(T, B, H, T, c.d), (left, 0)
    kw = dict(new_lens=None if new is None else i32(new), window=window)
    n_dev, page = i32(lens), c.page
    _, lse = fa.fwd_paged(q, c.k, c.v, table, n_dev, **kw)
    for b in range(B):
        if lens[b] > 0:
            c.forget(b, 0 if decay == 0 and fresh[b] else lens[b] - fresh[b], lens[b])
    before = c.w.clone()
    fa.kv_weights(q, lse, c.k, c.w, table, n_dev, decay=decay, **kw)
    torch.cuda.synchronize()
    assert fa.fa_fwd_status(None) == (0, 0)
    written = torch.zeros(c.w.shape, dtype=torch.bool, device="cuda")
    for b, (n, m) in enumerate(zip(lens, fresh)):
        if n <= 0 or m == 0:
            continue
        j = np.arange(n)
        pages, slots = torch.from_numpy(c.table[b][j // page]).long().cuda(), torch.from_numpy(j % page).cuda()
        for h in range(Hk):
            at, G = (pages, h, slots), H // Hk
            want, tol = definition(q[b, h * G:(h + 1) * G, :m], lse[b, h * G:(h + 1) * G, :m], c.k[at], before[at], n, m,
                                   left, decay)
            err = (c.w[at].double() - want).abs()
            assert bool((err <= tol).all()), f"sequence {b}, head {h}: off by {float(err.max()):.3e}"
            written[at] = True
    assert torch.equal(bits(c.w)[~written], bits(before)[~written])


@pytest.mark.parametrize("decay", [0.5, 0.0, 1.0])
@pytest.mark.parametrize("B,H,Hk,T,d,page,lens,new,left", roles.CASES)
def test_units_that_no_row_sees(fa, B, H, Hk, T, d, page, lens, new, left, decay):
    c = Cache(B + T, lens, Hk, d, page)
    check(fa, c, B, H, Hk, T, lens, new, left, decay, c.device_table())


@pytest.mark.parametrize("B,H,Hk,T,d,lens,new", [
    (4, 8, 4, 70, 64, [300, 0, -1, 5], [70, 0, 70, 5]),
    (3, 12, 2, 1300, 128, [0, 1300, 40], [0, 1300, 3]),  # by cost, or with as many CTAs to a unit as there are SMs for
    (2, 5, 5, 200, 128, [0, -2], [200, 0]),              # no unit at all
])
@pytest.mark.parametrize("width", [30, 900])
def test_clusters_without_a_unit(fa, B, H, Hk, T, d, lens, new, width):
    """A table for far longer sequences: most clusters of the launch find nothing to do."""
    c = Cache(B + T, lens, Hk, d, 64)
    table = np.full((B, width), -9, np.int32)
    table[:, :c.table.shape[1]] = c.table
    check(fa, c, B, H, Hk, T, lens, new, -1, 0.5, torch.from_numpy(table).cuda())
